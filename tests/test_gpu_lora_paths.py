"""The adapters' kernels for many rows, which a short call's one launch never
reaches: every block of ranks, tiles of 64 and of 128 rows, several slices of K
and pieces of every length, with the tolerances of the operators' own tests;
the sizes on both sides of each rule; gradients of longer groups exactly, on
small integers whose sums fp32 holds in any order.

Each case says which kernels it is for, and fails where a changed rule takes it
elsewhere."""
import ctypes

import numpy as np
import pytest

from tests.gpu_util import dev_bits, dev_i32, empty_bits
from tests.test_gpu_lora import G, Case, backward, bits, check_behind, forward, workspace  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
ONE, FEW, MB1, MB2 = 0, 1, 2, 3


def takes(G, M, L, r, K, N):  # noqa: F811
    out = (ctypes.c_int * 3)()
    G._lib.moe_lora_takes(M, L, r, K, N, out)
    return tuple(out)


# counts, T, r, K, N, (forward, backward, rows of a piece)
PATHS = {
    "rank 8, many tiles": ([4000, 0, 170], 4200, 8, 264, 136, (MB2, MB2, 128)),
    "rank 16, uneven tiles of 64": ([60, 70, 0, 64, 66] * 18, 4700, 16, 136, 264, (MB1, MB1, 128)),
    "rank 24": ([170, 90], 270, 24, 5504, 264, (MB2, ONE, 128)),
    "rank 24, wide": ([170, 90], 270, 24, 264, 5504, (ONE, MB2, 128)),
    "rank 32, tiles of 64": ([100, 65, 0, 110], 280, 32, 4104, 4168, (MB1, MB1, 128)),
    "rank 32, tiles of 128": ([128, 172], 300, 32, 4200, 4104, (MB2, MB2, 128)),
    "rank 40, tiles of 64": ([0, 129, 64, 90], 290, 40, 3288, 72, (MB1, MB1, 128)),
    "rank 64, tiles of 128": ([257, 43], 310, 64, 2056, 776, (MB2, MB2, 128)),
    "rank 64, many rows": ([1501, 0, 640], 2150, 64, 520, 1032, (MB2, MB2, 128)),
    "rank 72, tiles of 128": ([300, 1], 305, 72, 1832, 520, (MB2, MB2, 128)),
    "rank 128, tiles of 64": ([65, 100, 0, 127], 295, 128, 1032, 392, (MB1, MB1, 128)),
    "rank 128, many rows": ([900, 1300], 2200, 128, 264, 520, (MB2, MB2, 128)),
    "pieces of 192": ([7001, 0, 1999], 9000, 16, 2056, 1032, (MB2, MB2, 192)),
    "pieces of 256, rank 96": ([4000, 193, 807], 5000, 96, 2312, 2056, (MB2, MB2, 256)),
    "90 groups": ([66, 0, 53, 71, 1, 90] * 15, 4300, 16, 136, 72, (MB1, MB1, 128)),
    "few rows of many groups": ([3, 0, 4, 5] * 75, 910, 16, 136, 264, (FEW, MB1, 128)),
    "few rows of many groups, rank 24": ([3, 0, 4, 5] * 75, 910, 24, 512, 72, (FEW, MB1, 128)),
    "few rows of many groups, rank 40": ([1, 0, 17, 2] * 60, 1200, 40, 264, 136, (MB1, MB1, 128)),
    "few rows of many groups, rank 64": ([1, 0, 9, 2] * 60, 720, 64, 504, 136, (FEW, MB1, 128)),
    "few rows of many groups, rank 128": ([1, 0, 2, 5] * 60, 500, 128, 520, 72, (FEW, MB1, 128)),
    "1000 groups": ([5, 0, 6, 7, 3] * 200, 4300, 8, 72, 136, (MB1, MB1, 128)),
}


def make(name, seed, **kw):
    counts, T, r, K, N, _ = PATHS[name]
    return Case(seed, counts, T, r, K, N, **kw)


@pytest.mark.parametrize("name", list(PATHS))
@pytest.mark.parametrize("direct", [False, True])
def test_forward(G, name, direct):  # noqa: F811
    c = make(name, 21, direct=direct)
    assert takes(G, c.M_cap, c.L, c.r, c.K, c.N) == PATHS[name][5]
    forward(G, c)
    forward(G, c, base="same", keep_u=False)
    forward(G, c, base=None)
    forward(G, c, base=None, keep_u=False)


@pytest.mark.parametrize("name", list(PATHS))
@pytest.mark.parametrize("direct", [False, True])
def test_backward(G, name, direct):  # noqa: F811
    c = make(name, 22, direct=direct)
    assert takes(G, c.M_cap, c.L, c.r, c.K, c.N) == PATHS[name][5]
    backward(G, c)
    backward(G, c, dx="same", accumulate=True)
    backward(G, c, dx=None, want_dB=False)


@pytest.mark.parametrize("name", ["rank 8, many tiles", "rank 32, tiles of 64", "rank 64, tiles of 128", "rank 128, tiles of 64"])
def test_src_outside(G, name):  # noqa: F811
    c = make(name, 23, outside=40)
    forward(G, c)
    forward(G, c, base="same")
    backward(G, c)
    backward(G, c, dx="same", accumulate=True)
    counts, T, r, K, N, _ = PATHS[name]
    c = Case(24, counts, T // 2, r, K, N, direct=True)       # grouped rows past the rows of x
    c.M_cap = int(sum(counts)) + 90                          # and a capacity past the groups
    forward(G, c)
    backward(G, c)


@pytest.mark.parametrize("name", ["rank 16, uneven tiles of 64", "rank 32, tiles of 128", "rank 64, tiles of 128", "rank 128, tiles of 64"])
def test_row_distances(G, name):  # noqa: F811
    _, _, _, K, N, _ = PATHS[name]
    c = make(name, 25, x_ld=K + 24, y_ld=2 * N)
    forward(G, c)
    forward(G, c, base="same")
    backward(G, c)
    backward(G, c, dx="same", accumulate=True)


# M, L, r, K: one row fewer takes the path before, this many the one after
BORDERS = [(4096, 1, 8, 264, MB2), (4080, 2, 32, 264, MB2), (2048, 1, 40, 136, MB2), (1024, 1, 128, 72, MB2), (1008, 2, 72, 72, MB2)]


@pytest.mark.parametrize("M,L,r,K,after", BORDERS)
def test_sides_of_one_launch(G, M, L, r, K, after):  # noqa: F811
    for m, want in ((M - 1, ONE), (M, after)):
        counts = [m] if L == 1 else [m - 17] + [0] * (L - 2) + [17]
        assert takes(G, m, L, r, K, 136)[0] == want, m
        c = Case(26, counts, m, r, K, 136)
        forward(G, c)
        backward(G, c)


@pytest.mark.parametrize("r,K", [(8, 16384), (32, 4096), (64, 2048), (128, 1024)])
def test_longest_weights_of_one_launch(G, r, K):  # noqa: F811
    for k, want in ((K, ONE), (K + 8, FEW)):
        assert takes(G, 40, 3, r, k, 136)[0] == want
        forward(G, Case(27, [20, 0, 20], 44, r, k, 136))
    if r <= 32:
        for n, want in ((K, ONE), (K + 8, MB1)):
            assert takes(G, 40, 3, r, 136, n)[1] == want
            backward(G, Case(28, [20, 0, 20], 44, r, 136, n))


@pytest.mark.parametrize("name", ["rank 8, many tiles", "rank 24", "rank 24, wide", "rank 32, tiles of 64", "rank 64, many rows",
                                  "rank 128, many rows", "90 groups"])
def test_same_bits_again(G, name):  # noqa: F811
    """Eagerly, from a replayed graph and beside another stream's work."""
    import torch
    c = make(name, 29)
    T, r = c.T, c.r
    grp, lo, src = c.group(G), c.lora(G), dev_i32(c.src)
    x, dy, base = dev_bits(c.x), dev_bits(c.dy), dev_bits(c.base)

    def buffers():
        need = max(G.moe_lora_fwd_workspace_bytes(c.M_cap, c.L, r, c.K, c.N), G.moe_lora_bwd_workspace_bytes(c.M_cap, c.L, r, c.K, c.N))
        return dict(y=empty_bits((T, c.N)), u=torch.zeros(c.M_cap, r, device="cuda"), dx=empty_bits((T, c.K)),
                    dA=torch.empty(c.L, r, c.K, device="cuda"), dB=torch.empty(c.L, c.N, r, device="cuda"), ws=workspace(need))

    def go(b, s=None):
        G.moe_lora_fwd(x, T, grp, lo, b["y"], base=base, src=src, u=b["u"], workspace=b["ws"], stream=s)
        G.moe_lora_bwd(dy, x, T, grp, lo, b["u"], dx=b["dx"], dA=b["dA"], dB=b["dB"], src=src, workspace=b["ws"], stream=s)

    def read(b):
        torch.cuda.synchronize()
        check_behind(b["ws"])
        return [b[k].cpu().numpy().tobytes() for k in ("y", "u", "dx", "dA", "dB")]
    first = buffers()
    go(first)
    want = read(first)
    for k in ("y", "u", "dx", "dA", "dB"):
        first[k].zero_()
    first["y"].copy_(empty_bits((T, c.N)))
    first["dx"].copy_(empty_bits((T, c.K)))
    go(first)
    assert read(first) == want
    graphed, side = buffers(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        go(graphed, side.cuda_stream)
    torch.cuda.synchronize()
    for _ in range(3):
        for k in ("u", "dA", "dB"):
            graphed[k].fill_(5.0)
        graphed["u"].zero_()
        torch.cuda.synchronize()
        g.replay()
        assert read(graphed) == want
    both, streams = [buffers(), buffers()], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for b, s in zip(both, streams):
            go(b, s.cuda_stream)
    torch.cuda.synchronize()
    assert read(both[0]) == want and read(both[1]) == want


@pytest.mark.parametrize("r", [8, 16, 32, 64])
def test_long_pieces_exactly(G, r):  # noqa: F811
    """Groups of several pieces of 1024 rows.  dy, B, x and u are small integers, so that w and every sum are whole
    numbers below 2^24: a row lost or counted twice shows in whichever order they are added."""
    import torch
    M, K, N = 17000, 7168, 7168
    counts = [12001, 3, 0, 4990]
    L = len(counts)
    assert takes(G, M, L, r, K, N)[2] == 1024
    gen = torch.Generator(device="cuda").manual_seed(30)
    ints = lambda n, *s: torch.randint(-n, n + 1, s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    x, A, B = ints(1, M, K), ints(1, L, r, K), ints(1, L, N, r)
    dy = ints(1, M, N)
    dy[:, 64:] = 0                                            # |w| <= 64: sums of 12001 rows stay below 2^20
    dy[:, 5000] = 1
    u = torch.randint(-9, 10, (M, r), generator=gen, device="cuda").float()
    src = torch.randperm(M, generator=gen, device="cuda").int()
    dA, dB = torch.full((L, r, K), 3.0, device="cuda"), torch.full((L, N, r), 3.0, device="cuda")
    ws = workspace(G.moe_lora_bwd_workspace_bytes(M, L, r, K, N))
    grp = G.groups(torch.tensor(counts, dtype=torch.int32, device="cuda"), M)
    dx = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    G.moe_lora_bwd(dy, x, M, grp, G.lora(A, B, r, K, N), u, dx=dx, dA=dA, dB=dB, accumulate=True, src=src, workspace=ws)
    torch.cuda.synchronize()
    check_behind(ws)
    at = 0
    for e, m in enumerate(counts):
        rows = src[at:at + m].long()
        d, X, U = dy[rows].float(), x[rows].float(), u[at:at + m]
        w = d @ B[e].float()                                  # exact in fp32, as are the sums
        assert torch.equal(dA[e].double(), w.double().t() @ X.double() + 3), e
        assert torch.equal(dB[e].double(), d.double().t() @ U.double() + 3), e
        at += m
