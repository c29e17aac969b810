"""The MXFP4 products at the ends of their documented sizes: the longest rows (a
tile's 256 rows of e4m3 codes reach almost 2^32 bytes), the widest outputs (256
rows of them too), and 1024 experts, on both kernels.  On small integers, whose
sums are exact, so that outputs are the nearest bf16; or with the tolerances of
test_gpu_mxfp4."""
import numpy as np
import pytest

from tests.gpu_util import BF16_NAN_SENTINEL, dev_i32, empty_bits
from tests.test_gpu_mxfp4 import G, _check, _operands, _product  # noqa: F401  (G: the fixture)
from tests.test_gpu_mxfp4_tiles import on_tiles

pytestmark = pytest.mark.gpu
E2M1 = {0: 0.0, 1: 0.5, 2: 1.0, 8: -0.0, 9: -0.5, 10: -1.0}
E4M3 = {0: 0.0, 0x30: 0.5, 0x38: 1.0, 0x80: -0.0, 0xB0: -0.5, 0xB8: -1.0}


def _codes(table, *shape, seed=0):
    """Random codes of 0, +-0.5 and +-1 on the GPU."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.tensor(list(table), dtype=torch.uint8, device="cuda")
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for part in out.view(-1).split(1 << 28):
        part.copy_(t[torch.randint(0, 6, part.shape, generator=g, device="cuda", dtype=torch.uint8).int()])
    return out


def _nibbles(*shape, seed=1):
    q = _codes(E2M1, *shape, seed=seed)
    q |= _codes(E2M1, *shape, seed=seed + 1) << 4
    return q


def _values(codes, fp4):
    """float64 values of a few rows of codes."""
    import torch
    table = torch.zeros(256, dtype=torch.float64, device="cuda")
    for c, v in (E2M1 if fp4 else E4M3).items():
        table[c] = v
    if fp4:
        codes = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    return table[codes.int()]


def _ones(*shape):
    import torch
    return torch.full(shape, 127, dtype=torch.uint8, device="cuda")


def _run(G, aq, bq, M, N, K, a, margin):  # noqa: F811
    import torch
    out = empty_bits((M + 1, N))
    A = G.operand(aq, dtype=G.DT_MXFP4 if a == "fp4" else G.DT_MXFP8, scales=_ones(M, K // 32))
    B = G.operand(bq, dtype=G.DT_MXFP4, layout=G.B_NK, scales=_ones(1, N, K // 32))
    G.moe_group_gemm_quant(A, B, N, K, G.groups(dev_i32([M]), M), out, cu_margin=margin)
    torch.cuda.synchronize()
    assert bool((out[M] == int(np.uint16(BF16_NAN_SENTINEL).view(np.int16))).all())
    return out.view(torch.bfloat16)[:M]


@pytest.mark.parametrize("a", ["fp4", "fp8"])
def test_longest_rows(G, a):  # noqa: F811
    import torch
    M, N, K = 300, 64, (1 << 24) - 32
    aq = _nibbles(M, K // 2) if a == "fp4" else _codes(E4M3, M, K)
    bq = _nibbles(1, N, K // 2, seed=3)
    rows, cols = [0, 1, 254, 255, 256, 299], [0, 1, 31, 62, 63]
    want = torch.zeros(len(rows), len(cols), dtype=torch.float64, device="cuda")
    step = 1 << 21
    for k in range(0, K, step):
        k1 = min(K, k + step)
        av = _values(aq[rows, k // 2:k1 // 2] if a == "fp4" else aq[rows, k:k1], a == "fp4")
        want += av @ _values(bq[0, cols, k // 2:k1 // 2], True).t()
    want = want.to(torch.bfloat16)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    margin = min(m for m in range(cus) if on_tiles(G, M, 1, N, K, a, m))      # (a few units have to do)
    assert margin > 0
    for m in (0, margin):                                                     # streamed; tiles
        got = _run(G, aq, bq, M, N, K, a, m)
        assert torch.equal(got[rows][:, cols], want), m


@pytest.mark.parametrize("a", ["fp4", "fp8"])
@pytest.mark.parametrize("M", [5, 300])                  # streamed; tiles
def test_widest_outputs(G, a, M):  # noqa: F811
    import torch
    N, K = (1 << 23) - 64, 32
    assert on_tiles(G, M, 1, N, K, a) == (M == 300)
    aq = _nibbles(M, K // 2) if a == "fp4" else _codes(E4M3, M, K)
    bq = _nibbles(1, N, K // 2, seed=3)
    got = _run(G, aq, bq, M, N, K, a, 0)
    av = _values(aq, a == "fp4")
    for c0 in (0, 1 << 22, N - 700):
        want = (av @ _values(bq[0, c0:c0 + 700], True).t()).to(torch.bfloat16)
        assert torch.equal(got[:, c0:c0 + 700], want), c0


@pytest.mark.parametrize("a", ["fp4", "fp8"])
def test_many_experts_on_tiles(G, a):  # noqa: F811
    E, N, K = 1024, 320, 288
    rng = np.random.default_rng(5)
    counts = rng.integers(0, 130, E)
    counts[[0, 500, 1023]] = 0, 700, 257
    counts[7:40] = 0
    M = int(counts.sum())
    assert on_tiles(G, M + 3, E, N, K, a)
    ops = _operands(rng, M + 3, K, E, N, a)
    _check(_product(G, counts, M + 3, K, N, a, ops, scale_shift=1), counts, M, ops[4], ops[5], a)
