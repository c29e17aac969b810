"""The 256 x 256 tiles of the MXFP4 products, at sizes that are seen to reach
them.  Tolerances as in test_gpu_mxfp4."""
import numpy as np
import pytest

from oracle import moe as O
from oracle import operators as P
from tests.gpu_util import dev_bytes, dev_i32, empty_bits, host_bits
from tests.test_gpu_mxfp4 import G, _check, _operands, _product  # noqa: F401  (G: the fixture)
from tests.test_gpu_operators_large import _bytes, _tol, f64

pytestmark = pytest.mark.gpu


def on_tiles(G, M_cap, E, N, K, a, cu_margin=0):  # noqa: F811
    import torch
    cus = torch.cuda.get_device_properties(0).multi_processor_count - cu_margin
    return bool(G._lib.moe_mx4_takes_tiles(M_cap, E, N, K, int(a == "fp4"), cus))


# m-tiles of up to 128 rows and of more in turn, which store different numbers of rows; groups without rows; N that
# ends inside a tile, so that some waves store nothing
STREAM = [700, 100, 5, 1513, 0, 128, 129, 1700, 1, 1257]


@pytest.mark.parametrize("a", ["fp4", "fp8"])
@pytest.mark.parametrize("N,K", [(1984, 32), (1984, 64), (1984, 96), (1984, 160), (1984, 224), (704, 256), (832, 352),
                                 (704, 384), (832, 480), (704, 544), (832, 1056)])
def test_tiles_in_a_stream_repeat_their_bits(G, a, N, K):  # noqa: F811
    """Several tiles per workgroup, whose K-tiles are one stream over them, one round of K-tiles or several behind the
    last tile's stores; rows of fewer blocks than a round.  The same bits in every run, with other values in the
    outputs and other work before."""
    import torch
    rng = np.random.default_rng(N + K)
    M, E = sum(STREAM), len(STREAM)
    ops = _operands(rng, M, K, E, N, a)
    first = None
    for i in range(6):
        margin = 250 if i < 4 else 253
        assert on_tiles(G, M, E, N, K, a, margin)
        junk = torch.full(((1 + i) << 20,), i, device="cuda")
        got = _product(G, STREAM, M, K, N, a, ops, cu_margin=margin, scale_shift=i % 4)
        junk += 1
        if first is None:
            first = got
            _check(got, STREAM, M, ops[4], ops[5], a)
        assert np.array_equal(got, first), i


@pytest.mark.parametrize("a", ["fp4", "fp8"])
def test_tiles_status_of_bad_counts(G, a):  # noqa: F811
    import torch
    E, M_cap, N, K = 3, 2000, 576, 1056
    assert on_tiles(G, M_cap, E, N, K, a, 250)
    ops = _operands(np.random.default_rng(16), M_cap, K, E, N, a)
    half = M_cap // 2
    for counts, eff, st in (([half, 5, 0], [half, 5, 0], 0), ([half, -5, 4], [half, 0, 4], 1),
                            ([half, M_cap, 7], [half, M_cap - half, 0], 2),
                            ([-1, M_cap + 1, 7], [0, M_cap, 0], 3), ([1 << 30, 1 << 30, 1 << 30], [M_cap, 0, 0], 2),
                            ([0, 0, 0], [0, 0, 0], 0)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        offs = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
        got = _product(G, counts, M_cap, K, N, a, ops, status, offs, cu_margin=250)
        assert int(status) == st
        assert offs.tolist() == [0] + np.cumsum(eff).tolist()
        _check(got, eff, sum(eff), ops[4], ops[5], a)


@pytest.mark.parametrize("a", ["fp4", "fp8"])
def test_tiles_rows_do_not_depend_on_their_company(G, a):  # noqa: F811
    N, K, M = 128, 736, 3000
    assert on_tiles(G, M, 1, N, K, a, 250)
    ops = _operands(np.random.default_rng(8), M, K, 1, N, a)
    many = _product(G, [M], M, K, N, a, ops, cu_margin=250)
    turned = _product(G, [M], M, K, N, a, (np.roll(ops[0], 7, 0), np.roll(ops[1], 7, 0), ops[2], ops[3]), cu_margin=250)
    assert np.array_equal(np.roll(turned[:M], -7, 0), many[:M])
    _check(many, [M], M, ops[4], ops[5], a)


@pytest.mark.parametrize("a", ["fp4", "fp8"])
def test_tiles_of_weights_past_4_gib(G, a):  # noqa: F811
    """Weights of 4.4e9 bytes: the last experts' on the tiles."""
    import torch
    E, N, K, rows = 150, 8192, 7168, 3600
    assert on_tiles(G, rows, E, N, K, a)
    rng = np.random.default_rng(rows)
    b, bs = _bytes(E, N, K // 2), torch.full((E, N, K // 32), 120, dtype=torch.uint8, device="cuda")
    ac = rng.integers(0, 256, (rows, K // 2 if a == "fp4" else K)).astype(np.uint8)
    if a == "fp8":
        ac = np.where((ac & 0x7F) == 0x7F, ac & 0x80, ac)
    as_ = rng.integers(118, 124, (rows, K // 32)).astype(np.uint8)
    counts = np.zeros(E, np.int64)
    counts[[0, 146, 149]] = [1, rows // 2, rows - rows // 2 - 1]
    out = empty_bits((rows, N))
    A = G.operand(dev_bytes(ac), dtype=G.DT_MXFP4 if a == "fp4" else G.DT_MXFP8, scales=dev_bytes(as_))
    B = G.operand(b, dtype=G.DT_MXFP4, layout=G.B_NK, scales=bs)
    G.moe_group_gemm_quant(A, B, N, K, G.groups(dev_i32(counts), rows), out)
    got = f64(host_bits(out))
    av = P.mxfp4_dequantize_rows(ac, as_) if a == "fp4" else O.mx_dequantize_rows(ac, as_)
    cols = np.r_[0:16, N - 48:N]
    off = O.exclusive_offsets(counts)
    for e in (0, 146, 149):
        bv = P.mxfp4_dequantize_rows(b[e].cpu().numpy()[cols], bs[e].cpu().numpy()[cols])
        r = slice(int(off[e]), int(off[e + 1]))
        want, mag = av[r] @ bv.T, np.abs(av[r]) @ np.abs(bv).T
        assert np.all(np.abs(got[r][:, cols] - want) <= _tol(a, K, want, mag)), e
    del b, bs, B
    torch.cuda.empty_cache()


@pytest.mark.parametrize("a", ["fp4", "fp8"])
def test_the_listed_sizes_of_many_rows_are_on_tiles_and_few_are_not(G, a):  # noqa: F811
    assert on_tiles(G, 32768, 32, 5760, 2880, a) and on_tiles(G, 16384, 32, 4096, 7168, a)
    assert not on_tiles(G, 8, 32, 7168, 2048, a) and not on_tiles(G, 32, 32, 5760, 2880, a)
    # 16 scales are loaded at once: fewer are never on the tiles
    for cus in (1, 256):
        assert G._lib.moe_mx4_takes_tiles(15, 1, 64, 32, 1, cus) == 0 and G._lib.moe_mx4_takes_tiles(0, 1, 64, 32, 0, cus) == 0
