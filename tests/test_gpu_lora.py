"""The adapters' products and gradients on the GPU against the float64 oracle.

Tolerances, U = 2^-24.  A sum of n fp32 terms in any order is off by at most n U
times the sum of the terms' sizes; products of two bf16 values are exact in fp32.
  u, w: (K + 8) U sum |x| |A|.
  y, dx: the product with the weight takes u to 2^-17 of its value and adds 2 r
         terms: (2^-17 + (2 r + 8) U) s sum |u| |B|, what u itself is off by, and
         half a bf16 step, 2^-8 of the value.
  dA, dB: products of fp32 and bf16 values to 2^-24, added over a group's rows in
         three parts each: (3 m + 16) U s sum |w| |x|, and what w is off by.
Values below 1e-37, where bf16 and fp32 have no full precision, add 1e-37."""
import numpy as np
import pytest

import workloads as W
from oracle import formats as F
from oracle import training as P
from tests.gpu_util import BF16_NAN_SENTINEL, dev_bits, dev_i32, empty_bits, host_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = 1e-37


@pytest.fixture(scope="module")
def G():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_gemm_glu_amd as G
    G.moe_init(0)
    return G


def bits(rng, *shape, std=1.0):
    return W.to_bf16_bits((rng.standard_normal(shape) * std).astype(np.float32))


class Case:
    """Inputs of one call: counts of the groups, T rows of x and y, grouped rows up to M_cap."""

    def __init__(self, seed, counts, T, r, K, N, M_cap=None, direct=False, scale=True, outside=0, x_ld=0, y_ld=0):
        rng = np.random.default_rng(seed)
        self.counts = np.asarray(counts, dtype=np.int32)
        total = int(np.maximum(self.counts, 0).sum())
        self.M_cap = total if M_cap is None else M_cap
        self.T, self.r, self.K, self.N, self.L = T, r, K, N, len(counts)
        self.src = None
        if not direct:
            self.src = np.full(self.M_cap, -1, dtype=np.int32)
            n = min(total, self.M_cap, T)
            self.src[:n] = rng.permutation(T)[:n]
            if outside:
                at = rng.permutation(n)[:outside]
                self.src[at] = rng.choice([-1, T, T + 7, -(1 << 31), (1 << 31) - 1], outside)
        self.x_ld, self.y_ld = x_ld or K, y_ld or N
        self.x, self.base = bits(rng, T, K), bits(rng, T, N, std=2.0)
        self.A, self.B = bits(rng, self.L, r, K, std=K ** -0.5), bits(rng, self.L, N, r, std=r ** -0.5)
        self.scale = (rng.random(self.L) + 0.5).astype(np.float32) if scale else None
        self.dy, self.dx_base = bits(rng, T, N, std=0.1), bits(rng, T, K, std=0.1)

    def wide(self, a, ld):
        """bf16 bits in rows ld apart, on the device."""
        out = empty_bits((max(1, self.T), ld))
        out[:self.T, :a.shape[1]] = dev_bits(a)
        return out

    def group(self, G, **kw):
        return G.groups(dev_i32(self.counts), self.M_cap, **kw)

    def lora(self, G):
        import torch
        s = None if self.scale is None else torch.from_numpy(self.scale).cuda()
        return G.lora(dev_bits(self.A), dev_bits(self.B), self.r, self.K, self.N, scale=s,
                      x_ld=0 if self.x_ld == self.K else self.x_ld, y_ld=0 if self.y_ld == self.N else self.y_ld)


def workspace(n):
    """Just as large as needed, with values that are not numbers in it and more of them behind."""
    import torch
    return torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")[:n]


def check_behind(ws):
    import torch
    whole = torch.empty(0, dtype=torch.uint8, device="cuda").set_(ws.untyped_storage())
    assert whole.numel() == ws.numel() + 4096 and torch.all(whole[ws.numel():] == 0xFF)


def check(got, want, tol, what):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(err / np.maximum(tol, 1e-300))), np.argwhere(bad)[:4])


def forward(G, c, base="other", keep_u=True, src=True):
    import torch
    grp, lo = c.group(G), c.lora(G)
    d_src = None if c.src is None else dev_i32(c.src)
    x = c.wide(c.x, c.x_ld)
    b = None if base is None else c.wide(c.base, c.y_ld)
    y = b if base == "same" else empty_bits((max(1, c.T), c.y_ld))
    u = torch.full((c.M_cap + 1, c.r), -7.0, device="cuda") if keep_u else None
    ws = workspace(G.moe_lora_fwd_workspace_bytes(c.M_cap, c.L, c.r, c.K, c.N))
    G.moe_lora_fwd(x, c.T, grp, lo, y, base=b, src=d_src, u=u, workspace=ws)
    torch.cuda.synchronize()
    check_behind(ws)
    got_u, got_y = None if u is None else u.cpu().numpy().astype(np.float64), host_bits(y)
    want_u, want_y = P.lora_fwd(c.x, c.A, c.B, c.scale, c.counts, c.M_cap, c.src, None if base is None else c.base)
    abs_s = None if c.scale is None else np.abs(c.scale)
    mag_u, _ = P.lora_fwd(c.x & 0x7FFF, c.A & 0x7FFF, c.B & 0x7FFF, abs_s, c.counts, c.M_cap, c.src)
    tol_u = (c.K + 8) * U * mag_u + TINY
    if keep_u:
        held = ~np.isnan(want_u[:, 0])
        check(got_u[:-1][held], want_u[held], tol_u[held], "u")
        assert np.all(got_u[:-1][~held] == -7) and np.all(got_u[-1] == -7)
    B = np.abs(F.bf16_bits_to_f64(c.B))
    tol_y = np.zeros((c.T, c.N))
    for e, g, rows in P.lora_rows(c.counts, c.M_cap, c.src, c.T):
        s = 1.0 if c.scale is None else abs(float(c.scale[e]))
        off = tol_u[g] + (2.0 ** -17 + (2 * c.r + 8) * U) * np.abs(want_u[g])
        tol_y[rows] = s * off @ B[e].T * 1.01
    written = ~np.isnan(want_y[:, 0]) if c.T else np.zeros(0, bool)
    g = F.bf16_bits_to_f64(got_y[:c.T, :c.N])
    check(g[written], want_y[written], (tol_y + 2.0 ** -8 * np.abs(want_y) * (1 + 2.0 ** -8) + TINY)[written], "y")
    untouched = c.base if base == "same" else np.full((c.T, c.N), BF16_NAN_SENTINEL, np.uint16)
    assert np.array_equal(got_y[:c.T, :c.N][~written], untouched[~written])
    assert np.all(got_y[:c.T, c.N:] == BF16_NAN_SENTINEL)      # between the rows
    return got_u, got_y


def backward(G, c, dx="other", want_dA=True, want_dB=True, accumulate=False):
    import torch
    grp, lo = c.group(G), c.lora(G)
    d_src = None if c.src is None else dev_i32(c.src)
    want_u, _ = P.lora_fwd(c.x, c.A, c.B, c.scale, c.counts, c.M_cap, c.src)
    u32 = np.nan_to_num(want_u, nan=3e38).astype(np.float32)    # rows of no group: never read
    x, dy = c.wide(c.x, c.x_ld), c.wide(c.dy, c.y_ld)
    base = None if dx in (None, "none") else c.wide(c.dx_base, c.x_ld)
    out = base if dx == "same" else None if dx is None else empty_bits((max(1, c.T), c.x_ld))
    start = 0.25 if accumulate else np.nan
    dA = torch.full((c.L, c.r, c.K), start, device="cuda") if want_dA else None
    dB = torch.full((c.L, c.N, c.r), start, device="cuda") if want_dB else None
    ws = workspace(G.moe_lora_bwd_workspace_bytes(c.M_cap, c.L, c.r, c.K, c.N))
    G.moe_lora_bwd(dy, x if want_dA else None, c.T, grp, lo, torch.from_numpy(u32).cuda() if want_dB else None, dx=out,
                   dx_base=base, dA=dA, dB=dB, accumulate=accumulate, src=d_src, workspace=ws)
    torch.cuda.synchronize()
    check_behind(ws)
    b = None if dx == "none" else c.dx_base
    want_dx, want_a, want_b, want_w = P.lora_bwd(c.dy, c.x, c.A, c.B, c.scale, c.counts, c.M_cap, u32, c.src, b)
    s_abs = None if c.scale is None else np.abs(c.scale)
    mag = lambda t: t & 0x7FFF  # noqa: E731
    _, mag_a, mag_b, mag_w = P.lora_bwd(mag(c.dy), mag(c.x), mag(c.A), mag(c.B), s_abs, c.counts, c.M_cap, np.abs(u32),
                                        c.src)
    tol_w = (c.N + 8) * U * mag_w + TINY
    A, ax = np.abs(F.bf16_bits_to_f64(c.A)), np.abs(F.bf16_bits_to_f64(c.x))
    tol_dx, off_a = np.zeros((c.T, c.K)), np.zeros(want_a.shape)
    for e, g, rows in P.lora_rows(c.counts, c.M_cap, c.src, c.T):
        s = 1.0 if c.scale is None else abs(float(c.scale[e]))
        tol_dx[rows] = s * (tol_w[g] + (2.0 ** -17 + (2 * c.r + 8) * U) * np.abs(want_w[g])) @ A[e] * 1.01
        off_a[e] = s * tol_w[g].T @ ax[rows] * 1.01
    m = np.array([len(g) for _, g, _ in P.lora_rows(c.counts, c.M_cap, c.src, c.T)])[:, None, None]
    add = start if accumulate else 0.0
    if want_dA:
        check(dA.cpu().numpy().astype(np.float64), want_a + add, (3 * m + 16) * U * (mag_a + add) + off_a + TINY, "dA")
    if want_dB:
        check(dB.cpu().numpy().astype(np.float64), want_b + add, (3 * m + 16) * U * (mag_b + add) + TINY, "dB")
    if out is not None:
        got = host_bits(out)
        written = ~np.isnan(want_dx[:, 0]) if c.T else np.zeros(0, bool)
        g = F.bf16_bits_to_f64(got[:c.T, :c.K])
        check(g[written], want_dx[written], (tol_dx + 2.0 ** -8 * np.abs(want_dx) * (1 + 2.0 ** -8) + TINY)[written], "dx")
        untouched = c.dx_base if dx == "same" else np.full((c.T, c.K), BF16_NAN_SENTINEL, np.uint16)
        assert np.array_equal(got[:c.T, :c.K][~written], untouched[~written])
        assert np.all(got[:c.T, c.K:] == BF16_NAN_SENTINEL)


CASES = {
    # counts, T, r, K, N
    "one row": ([1], 1, 8, 8, 8),
    "one token": ([0, 0, 1, 0], 1, 16, 512, 264),
    "few rows, many groups": ([1, 0, 3, 2, 0, 0, 5, 1], 17, 16, 264, 520),
    "tiles of 16": ([16, 17, 15, 0, 1], 50, 24, 136, 72),
    "tiles of 32": ([32, 33, 31, 64, 95], 260, 32, 640, 392),
    "rank 8": ([40, 3], 45, 8, 1032, 1160),
    "rank 40": ([70], 70, 40, 96, 200),
    "rank 64": ([9, 100], 110, 64, 1544, 136),
    "rank 120": ([37, 0, 20], 64, 120, 328, 1032),
    "rank 128": ([65, 130], 195, 128, 768, 384),
    "pieces": ([600, 0, 129, 128], 860, 16, 264, 136),
    "many rows, rank 8": ([1300, 0, 77], 1400, 8, 264, 392),
    "many rows, rank 16": ([2200], 2200, 16, 520, 1160),
    "many rows, rank 24": ([130, 700, 129, 640], 1600, 24, 776, 136),
    "many rows, rank 32": ([1, 900, 200, 300], 1500, 32, 1032, 1544),
    "many small groups": ([17, 3, 64, 65, 0, 30, 1, 20, 70, 66, 127, 128] * 4, 2400, 16, 392, 264),
    "many small groups, rank 24": ([17, 3, 64, 65, 0, 30, 1, 20, 70, 66, 100, 128] * 4, 2300, 24, 136, 520),
    "few rows, long": ([3, 0, 9, 16, 1, 17], 50, 16, 7168, 264),
    "few rows, long, rank 24": ([1, 0, 2, 5], 9, 24, 2888, 776),
    "one launch, rank 128": ([7, 30, 1, 0, 16], 60, 128, 512, 520),
    "one launch, rank 72": ([1, 17], 18, 72, 904, 264),
    "few rows, rank 16": ([1, 0, 17], 20, 16, 8200, 520),
    "few rows, rank 24, slices": ([2, 0, 5, 1], 9, 24, 5496, 136),
    "few rows, rank 64": ([3, 16], 21, 64, 2056, 264),
    "one launch, 200 tiles": ([17] * 90 + [0] * 20, 1600, 16, 264, 520),
    "one launch, rank 32": ([40, 3], 50, 32, 4096, 1032),
    "few rows, rank 128": ([7, 30, 1], 40, 128, 1032, 136),
    "one row in 100 groups, long": ([1] * 100, 100, 8, 8200, 72),
    "a tile more than one launch takes": ([2040], 2040, 8, 264, 136),
    "65 groups": ([i % 3 for i in range(65)], 70, 16, 72, 40),
    "1024 groups": ([1 if i % 11 == 5 else 0 for i in range(1024)], 100, 8, 64, 64),
}


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("direct", [False, True])
def test_forward(G, name, direct):
    counts, T, r, K, N = CASES[name]
    c = Case(1, counts, T, r, K, N, direct=direct)
    forward(G, c)
    forward(G, c, base="same", keep_u=False)
    forward(G, c, base=None)


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("direct", [False, True])
def test_backward(G, name, direct):
    counts, T, r, K, N = CASES[name]
    c = Case(2, counts, T, r, K, N, direct=direct)
    backward(G, c)
    backward(G, c, dx="same", accumulate=True)


def test_backward_parts(G):
    for direct in (False, True):
        c = Case(3, [150, 0, 41, 300], 500, 16, 1200, 1400, direct=direct)
        backward(G, c, dx=None)
        backward(G, c, dx="none", want_dA=False)
        backward(G, c, dx="other", want_dA=False, want_dB=False)
        backward(G, c, dx=None, want_dB=False)
        backward(G, c, dx=None, want_dA=False, accumulate=True)


def test_counts_that_do_not_fit(G):
    """Negative counts are none, counts past the capacity are cut; offsets and status say so."""
    import torch
    for counts, cap, status in (([5, -3, 20, 9], 40, 1), ([30, 30, 30], 50, 2), ([-1, 1 << 30, 1 << 30, 1 << 30], 33, 3),
                                ([0] * 70 + [9, -2, 70] + [1] * 30, 60, 3), ([7, 8], 15, 0)):
        c = Case(4, counts, 64, 16, 264, 72, M_cap=cap, direct=False)
        c.src = np.random.default_rng(1).permutation(64)[:cap].astype(np.int32)
        forward(G, c)
        backward(G, c)
        offs, st = torch.full((c.L + 1,), -7, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        grp = c.group(G, offsets_out=offs, status_out=st)
        y = empty_bits((64, c.N))
        G.moe_lora_fwd(dev_bits(c.x), 64, grp, c.lora(G), y, src=dev_i32(c.src),
                       workspace=workspace(G.moe_lora_fwd_workspace_bytes(cap, c.L, 16, c.K, c.N)))
        torch.cuda.synchronize()
        assert int(st) == status
        want = np.minimum(np.concatenate([[0], np.cumsum(np.maximum(counts, 0), dtype=np.int64)]), cap)
        assert offs.tolist() == want.tolist()


def test_src_outside(G):
    for name in ("tiles of 16", "tiles of 32", "rank 128", "pieces"):
        counts, T, r, K, N = CASES[name]
        c = Case(5, counts, T, r, K, N, outside=9)
        forward(G, c)
        forward(G, c, base="same")
        backward(G, c)
        c = Case(6, counts, max(1, T // 2), r, K, N, direct=True)   # grouped rows past the rows of x
        c.M_cap = T
        forward(G, c)
        backward(G, c)


def test_row_distances(G):
    for counts, T, r, K, N in (CASES["tiles of 32"], CASES["rank 8"]):
        c = Case(7, counts, T, r, K, N, x_ld=K + 24, y_ld=2 * N)
        forward(G, c)
        forward(G, c, base="same")
        backward(G, c)
        backward(G, c, dx="same", accumulate=True)


def test_no_scale(G):
    c = Case(8, [20, 33], 60, 16, 264, 136, scale=False)
    forward(G, c)
    backward(G, c)


def test_capacity_larger_than_the_rows(G):
    c = Case(9, [5, 0, 40, 1], 50, 16, 136, 72, M_cap=700)
    forward(G, c)
    backward(G, c)


def test_rows_stay_their_own(G):
    """A NaN or an infinity of one row, and of weights of a group without rows, reaches nothing else."""
    c = Case(10, [20, 30, 0], 60, 16, 264, 136)
    clean_u, clean_y = forward(G, c)
    bad = int(c.src[25])
    c.x[bad, 7], c.dy[bad, 5] = 0x7FC0, 0x7F80
    c.A[2], c.B[2] = 0x7FC0, 0x7F80
    import torch
    y, u = empty_bits((60, c.N)), torch.zeros(c.M_cap, c.r, device="cuda")
    ws = workspace(max(G.moe_lora_fwd_workspace_bytes(c.M_cap, c.L, c.r, c.K, c.N),
                       G.moe_lora_bwd_workspace_bytes(c.M_cap, c.L, c.r, c.K, c.N)))
    grp, lo, src = c.group(G), c.lora(G), dev_i32(c.src)
    G.moe_lora_fwd(dev_bits(c.x), 60, grp, lo, y, base=dev_bits(c.base), src=src, u=u, workspace=ws)
    dx, dA, dB = empty_bits((60, c.K)), torch.empty(3, c.r, c.K, device="cuda"), torch.empty(3, c.N, c.r, device="cuda")
    G.moe_lora_bwd(dev_bits(c.dy), dev_bits(c.x), 60, grp, lo, u, dx=dx, dA=dA, dB=dB, src=src, workspace=ws)
    torch.cuda.synchronize()
    got_y = host_bits(y)
    rest = np.arange(60) != bad
    assert np.array_equal(got_y[rest], clean_y[rest]) and np.all(np.isnan(F.bf16_bits_to_f64(got_y[bad])))
    assert np.all(np.isfinite(F.bf16_bits_to_f64(host_bits(dx)[c.src[:50]][np.arange(50) != 25])))
    assert torch.all(torch.isfinite(dA[0])) and torch.all(torch.isfinite(dB[0]))
    assert torch.all(torch.isnan(dA[1]).any(1)) and torch.all(dA[2] == 0) and torch.all(dB[2] == 0)


def test_infinite_u(G):
    """An infinite u is an infinity times the weights, not a NaN of its second part."""
    import torch
    c = Case(11, [3], 3, 8, 16, 8, scale=False)
    c.x[:], c.A[:], c.B[:] = 0x3F80, 0x3F80, 0x3F80            # 1
    c.x[1, 0] = 0x7F80
    y, u = empty_bits((3, 8)), torch.zeros(3, 8, device="cuda")
    G.moe_lora_fwd(dev_bits(c.x), 3, c.group(G), c.lora(G), y, u=u, src=dev_i32(c.src),
                   workspace=workspace(G.moe_lora_fwd_workspace_bytes(3, 1, 8, 16, 8)))
    torch.cuda.synchronize()
    got = F.bf16_bits_to_f64(host_bits(y))
    assert np.all(got[1] == np.inf) and np.all(got[[0, 2]] == 128)


def test_gradients_against_differences(G):
    """L = <dy, y>, on small integers that stay exact: the difference of two forward passes is the gradient."""
    import torch
    rng = np.random.default_rng(12)
    c = Case(12, [3, 5], 8, 8, 16, 8, scale=False)
    small = lambda *s: W.to_bf16_bits(rng.integers(-1, 2, s).astype(np.float32))  # noqa: E731
    c.x, c.A, c.B, c.dy = small(8, 16), small(2, 8, 16), small(2, 8, 8), small(8, 8)
    grp, src = c.group(G), dev_i32(c.src)
    ws = workspace(max(G.moe_lora_fwd_workspace_bytes(8, 2, 8, 16, 8), G.moe_lora_bwd_workspace_bytes(8, 2, 8, 16, 8)))

    def loss(x, A, B, u=None):
        y = empty_bits((8, 8))
        G.moe_lora_fwd(dev_bits(x), 8, grp, G.lora(dev_bits(A), dev_bits(B), 8, 16, 8), y, src=src, u=u, workspace=ws)
        torch.cuda.synchronize()
        return float(np.sum(F.bf16_bits_to_f64(host_bits(y)) * F.bf16_bits_to_f64(c.dy)))
    u = torch.zeros(8, 8, device="cuda")
    at = loss(c.x, c.A, c.B, u)
    dx, dA, dB = empty_bits((8, 16)), torch.empty(2, 8, 16, device="cuda"), torch.empty(2, 8, 8, device="cuda")
    G.moe_lora_bwd(dev_bits(c.dy), dev_bits(c.x), 8, grp, c.lora(G), u, dx=dx, dA=dA, dB=dB, src=src, workspace=ws)
    torch.cuda.synchronize()
    grads = {"x": F.bf16_bits_to_f64(host_bits(dx)), "A": dA.cpu().numpy(), "B": dB.cpu().numpy()}
    for name, g in grads.items():
        for _ in range(12):
            i = tuple(rng.integers(0, n) for n in g.shape)
            t = {k: getattr(c, k).copy() for k in ("x", "A", "B")}
            t[name][i] = W.to_bf16_bits(np.float32(F.bf16_bits_to_f64(t[name])[i] + 1).reshape(1))[0]
            assert loss(t["x"], t["A"], t["B"]) - at == g[i], (name, i)


def test_same_bits_again(G):
    """The order of every sum is fixed."""
    import torch
    c = Case(13, [700, 300, 0, 25], 1100, 32, 1032, 776)
    grp, lo, src = c.group(G), c.lora(G), dev_i32(c.src)
    got = []
    for _ in range(3):
        y, u = empty_bits((1100, c.N)), torch.zeros(c.M_cap, c.r, device="cuda")
        ws = workspace(max(G.moe_lora_fwd_workspace_bytes(c.M_cap, c.L, c.r, c.K, c.N),
                           G.moe_lora_bwd_workspace_bytes(c.M_cap, c.L, c.r, c.K, c.N)))
        G.moe_lora_fwd(dev_bits(c.x), 1100, grp, lo, y, base=dev_bits(c.base), src=src, u=u, workspace=ws)
        dx, dA, dB = empty_bits((1100, c.K)), torch.empty(4, 32, c.K, device="cuda"), torch.empty(4, c.N, 32, device="cuda")
        G.moe_lora_bwd(dev_bits(c.dy), dev_bits(c.x), 1100, grp, lo, u, dx=dx, dA=dA, dB=dB, src=src, workspace=ws)
        torch.cuda.synchronize()
        got.append([t.cpu().numpy().tobytes() for t in (y, u, dx, dA, dB)])
    assert got[0] == got[1] == got[2]


def test_no_rows(G):
    import torch
    E, r, K, N = 3, 16, 64, 72
    lo = G.lora(torch.zeros(E, r, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(E, N, r, dtype=torch.bfloat16, device="cuda"), r, K, N)
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    empty = torch.empty(0, K, dtype=torch.bfloat16, device="cuda")
    offs, st = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    G.moe_lora_fwd(empty, 0, G.groups(counts, 0, offsets_out=offs, status_out=st), lo, empty)
    dA, dB = torch.full((E, r, K), 5.0, device="cuda"), torch.full((E, N, r), 5.0, device="cuda")
    G.moe_lora_bwd(empty, empty, 0, G.groups(counts, 0), lo, None, dx=empty, dA=dA, dB=dB, accumulate=True)
    torch.cuda.synchronize()
    assert offs.tolist() == [0] * 4 and torch.all(dA == 5) and torch.all(dB == 5)
    G.moe_lora_bwd(empty, empty, 0, G.groups(counts, 0), lo, None, dx=empty, dA=dA, dB=dB)
    torch.cuda.synchronize()
    assert torch.all(dA == 0) and torch.all(dB == 0)
    # rows, but of no group
    x, y = torch.ones(9, K, dtype=torch.bfloat16, device="cuda"), torch.ones(9, N, dtype=torch.bfloat16, device="cuda")
    ws = workspace(G.moe_lora_bwd_workspace_bytes(9, E, r, K, N))
    u = torch.full((9, r), float("nan"), device="cuda")
    G.moe_lora_fwd(x, 9, G.groups(counts, 9), lo, y, u=u, workspace=ws)
    dA.fill_(5), dB.fill_(5)
    G.moe_lora_bwd(y, x, 9, G.groups(counts, 9), lo, u, dA=dA, dB=dB, workspace=ws)
    torch.cuda.synchronize()
    assert torch.all(y == 1) and torch.all(torch.isnan(u)) and torch.all(dA == 0) and torch.all(dB == 0)
