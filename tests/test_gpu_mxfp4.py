"""MXFP4 quantisation and the grouped products with MXFP4 weights on the GPU
against the float64 oracle.

Tolerances.  Codes and scales are equal byte for byte.  Products, u = 2^-24: of
4-bit rows, a step of 128 products is summed by the MFMA to 4 u of the sum of
their sizes, the steps and the waves' shares in fp32: (K / 128 + 16) 4 u of the
sum of the products' sizes; of 8-bit rows MX_ACC_REL (gpu_util) of it, the
block-scaled MFMA's own accumulation; then half a bf16 step (2^-8).  On small
integers every sum is exact."""
import numpy as np
import pytest

import workloads as W
from oracle import formats as F
from oracle import moe as O
from oracle import operators as P
from tests.gpu_util import (BF16_NAN_SENTINEL, BYTE_SENTINEL, MX_ACC_REL, dev_bits, dev_bytes, dev_i32, empty_bits,
                            empty_bytes, host_bits)

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def G():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_gemm_glu_amd as G
    G.moe_init(0)
    return G


def _wide(rng, R, C):
    """bf16 values whose 32-blocks differ in size by powers of two."""
    v = rng.standard_normal((R, C)) * np.exp2(rng.integers(-8, 8, (R, C // 32))).repeat(32, 1)
    return W.to_bf16_bits(v.astype(np.float32))


# ---------------------------------------------------------------- quantisation
@pytest.mark.parametrize("R,C", [(1, 32), (3, 64), (17, 96), (5, 2880), (40, 7168), (1000, 160)])
def test_quantize_rows(G, R, C):
    import torch
    v = _wide(np.random.default_rng(R + C), R, C)
    q, s = empty_bytes((R + 1, C // 2)), empty_bytes((R + 1, C // 32))
    G.moe_mxfp4_quantize(dev_bits(v), R, C, None, q, s)
    torch.cuda.synchronize()
    rq, rs = P.mxfp4_quantize_rows(v)
    qh, sh = q.cpu().numpy(), s.cpu().numpy()
    assert np.array_equal(sh[:R], rs) and np.array_equal(qh[:R], rq)
    assert np.all(qh[R] == BYTE_SENTINEL) and np.all(sh[R] == BYTE_SENTINEL)


def test_quantize_every_bf16_value(G):
    """Each of the 65536 bf16 patterns beside each of a few block maxima."""
    import torch
    bits = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    tops = np.array([0x40C0, 0x40C1, 0x3F80, 0x0001, 0x0080, 0x7F7F, 0x4040, 0x7F40], dtype=np.uint16)
    v = np.zeros((len(tops), 1 << 16, 1), np.uint16)
    v[:, :, 0] = bits
    v = v.reshape(len(tops), -1, 8)                         # 8 patterns, the maximum, zeros
    v = np.concatenate([v, np.broadcast_to(tops[:, None, None], v.shape[:2] + (1,)),
                        np.zeros(v.shape[:2] + (23,), np.uint16)], axis=2).reshape(-1, 32)
    q, s = empty_bytes((len(v), 16)), empty_bytes((len(v), 1))
    G.moe_mxfp4_quantize(dev_bits(v), len(v), 32, None, q, s)
    torch.cuda.synchronize()
    rq, rs = P.mxfp4_quantize_rows(v)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


def test_quantize_routed_rows_only(G):
    import torch
    R, C = 50, 64
    v = _wide(np.random.default_rng(1), R, C)
    rq, rs = P.mxfp4_quantize_rows(v)
    for counts, n in (([3, 0, 20], 23), ([0, 0], 0), ([30, 40], 50), ([-4, 7], 7)):
        q, s = empty_bytes((R, C // 2)), empty_bytes((R, C // 32))
        G.moe_mxfp4_quantize(dev_bits(v), R, C, G.groups(dev_i32(counts), R), q, s)
        torch.cuda.synchronize()
        qh, sh = q.cpu().numpy(), s.cpu().numpy()
        assert np.array_equal(qh[:n], rq[:n]) and np.array_equal(sh[:n], rs[:n])
        assert np.all(qh[n:] == BYTE_SENTINEL) and np.all(sh[n:] == BYTE_SENTINEL)


@pytest.mark.parametrize("E,N,K", [(1, 64, 32), (3, 192, 96), (2, 320, 544)])
def test_pack_weight(G, E, N, K):
    import torch
    w = _wide(np.random.default_rng(N + K), E * N, K).reshape(E, N, K)
    w[0, 1, 3], w[0, 2, 4] = 0x7FC0, 0xFF80
    rq, rs = P.mxfp4_quantize_rows(w.reshape(E * N, K))
    for layout, src in ((G.B_NK, w), (G.B_KN, np.ascontiguousarray(w.transpose(0, 2, 1)))):
        q, s = empty_bytes((E * N + 1, K // 2)), empty_bytes((E * N + 1, K // 32))
        G.moe_pack_weight_mxfp4(dev_bits(src), E, N, K, layout, q, s)
        torch.cuda.synchronize()
        qh, sh = q.cpu().numpy(), s.cpu().numpy()
        assert np.array_equal(sh[:-1], rs) and np.array_equal(qh[:-1], rq)
        assert np.all(qh[-1] == BYTE_SENTINEL) and np.all(sh[-1] == BYTE_SENTINEL)


# ---------------------------------------------------------------- product
def _operands(rng, M_cap, K, E, N, a, wide=True):
    """Codes and scales of rows and weights, with their float64 values."""
    ac = rng.integers(0, 256, (M_cap, K // 2 if a == "fp4" else K)).astype(np.uint8)
    if a == "fp8":
        ac = np.where((ac & 0x7F) == 0x7F, ac & 0x80, ac)          # no NaN codes
    sc = (lambda *n: rng.integers(118, 130, n).astype(np.uint8)) if wide else (lambda *n: np.full(n, 127, np.uint8))
    as_, bs = sc(M_cap, K // 32), sc(E, N, K // 32)
    bc = rng.integers(0, 256, (E, N, K // 2)).astype(np.uint8)
    av = P.mxfp4_dequantize_rows(ac, as_) if a == "fp4" else O.mx_dequantize_rows(ac, as_)
    return ac, as_, bc, bs, av, P.mxfp4_dequantize_rows(bc, bs)


def _product(G, counts, M_cap, K, N, a, ops, status=None, offsets=None, cu_margin=0, scale_shift=0):
    import torch
    ac, as_, bc, bs = ops[:4]
    out = empty_bits((M_cap + 1, N))

    def scales(x):                          # at any address
        buf = empty_bytes((x.size + 16,))
        v = buf[scale_shift:scale_shift + x.size]
        v.copy_(dev_bytes(x.reshape(-1)))
        return v
    A = G.operand(dev_bytes(ac), dtype=G.DT_MXFP4 if a == "fp4" else G.DT_MXFP8, scales=scales(as_))
    B = G.operand(dev_bytes(bc), dtype=G.DT_MXFP4, layout=G.B_NK, scales=scales(bs))
    grp = G.groups(dev_i32(counts), M_cap, offsets_out=offsets, status_out=status)
    G.moe_group_gemm_quant(A, B, N, K, grp, out, cu_margin=cu_margin)
    torch.cuda.synchronize()
    return host_bits(out)


def _check(got, counts, M, av, bv, a, what=""):
    want, mag = P.group_gemm_values(av[:M], counts, bv)
    assert np.all(got[M:] == BF16_NAN_SENTINEL), f"{what}: rows behind the last group written"
    K = av.shape[1]
    acc = (K / 128 + 16) * 4 * U if a == "fp4" else MX_ACC_REL
    err = np.abs(F.bf16_bits_to_f64(got[:M]) - want)
    tol = 2.0 ** -8 * np.abs(want) + acc * mag + 1e-37
    assert np.all(err <= tol), (what, float(np.max(err / tol)))


CASES = [([1], 64, 32, 0), ([1, 0, 1], 64, 64, 3), ([0, 0], 64, 96, 2), ([2, 17, 0, 33], 128, 160, 0),
         ([64, 65, 1], 192, 256, 5), ([5, 3], 320, 288, 0), ([16, 15, 130, 0, 7], 64, 2880, 1),
         ([300, 0, 257, 1], 320, 544, 9), ([256, 512], 256, 512, 0), ([1, 2, 1, 0, 3, 1], 576, 7168, 0),
         ([700], 704, 384, 4), ([129, 255, 128], 512, 1056, 0)]


@pytest.mark.parametrize("a", ["fp4", "fp8"])
@pytest.mark.parametrize("counts,N,K,pad", CASES)
def test_product(G, counts, N, K, pad, a):
    rng = np.random.default_rng(N + K + sum(counts))
    M = sum(counts)
    ops = _operands(rng, M + pad, K, len(counts), N, a)
    got = _product(G, counts, M + pad, K, N, a, ops, scale_shift=K % 3)
    _check(got, counts, M, ops[4], ops[5], a)


@pytest.mark.parametrize("a", ["fp4", "fp8"])
@pytest.mark.parametrize("counts,N,K", [([40, 0, 300], 192, 352), ([3, 1], 64, 2048)])
def test_product_exact_on_small_integers(G, counts, N, K, a):
    """Codes 0, +-0.5, +-1 and scale 1: every sum is a multiple of 1/4 below
    2^22; outputs whose exact value is a bf16 are bit-exact, the others the
    nearest bf16."""
    rng = np.random.default_rng(K)
    M, E = sum(counts), len(counts)
    small = np.array([0, 1, 2, 8, 9, 10], np.uint8)

    def nibbles(*n):
        x = small[rng.integers(0, 6, n)]
        return x[..., 0::2] | (x[..., 1::2] << 4)
    bc, bs = nibbles(E, N, K), np.full((E, N, K // 32), 127, np.uint8)
    as_ = np.full((M, K // 32), 127, np.uint8)
    if a == "fp4":
        ac = nibbles(M, K)
        av = P.mxfp4_dequantize_rows(ac, as_)
    else:
        ac = np.array([0, 0x30, 0x38, 0x80, 0xB0, 0xB8], np.uint8)[rng.integers(0, 6, (M, K))]
        av = O.mx_dequantize_rows(ac, as_)
    bv = P.mxfp4_dequantize_rows(bc, bs)
    got = _product(G, counts, M, K, N, a, (ac, as_, bc, bs))
    want, _ = P.group_gemm_values(av, counts, bv)
    w = F.f64_to_bf16_bits(want)
    g = got[:M]
    assert np.array_equal(np.where(g == 0x8000, 0, g), np.where(w == 0x8000, 0, w))


@pytest.mark.parametrize("a", ["fp4", "fp8"])
def test_product_scale_extremes_and_nan(G, a):
    """The scales' whole range, a NaN scale in a row and in a weight, and a NaN
    row behind the groups that nothing may read."""
    rng = np.random.default_rng(5)
    counts, N, K = [20, 3], 64, 320
    M = 23
    ops = list(_operands(rng, M + 1, K, 2, N, a))
    ac, as_, bc, bs = ops[:4]
    as_[0], bs[0, 0] = 0, 254            # 2^-127 x 2^127
    as_[1, 2] = 255                      # row 1 is NaN everywhere
    bs[1, 5, 9] = 255                    # column 5 of group 1
    as_[2, :], bs[0, 1, :] = 254, 254    # beyond fp32: infinite, or NaN where both signs meet
    as_[M] = 255
    got = F.bf16_bits_to_f64(_product(G, counts, M + 1, K, N, a, ops))
    av = P.mxfp4_dequantize_rows(ac, as_) if a == "fp4" else O.mx_dequantize_rows(ac, as_)
    _, mag = P.group_gemm_values(av[:M], counts, P.mxfp4_dequantize_rows(bc, bs))
    nan = np.isnan(got[:M])
    assert np.all(nan[1]) and np.all(nan[20:, 5]) and np.all(~np.isfinite(got[2, 1]))
    assert np.all(nan[np.isnan(mag)])
    # a number elsewhere, unless the sum of the products' sizes passes fp32's range (the scales of 2^127 reach
    # every row of column 0 and 1 and every column of row 2)
    assert not np.any(nan & (mag < 2.0 ** 127))
    assert np.sum(mag < 2.0 ** 127) > M * N // 2 and mag[0, 0] < 2.0 ** 127
    want = av[0] @ P.mxfp4_dequantize_rows(bc, bs)[0, 0]
    assert abs(got[0, 0] - want) <= 2.0 ** -8 * abs(want) + MX_ACC_REL * mag[0, 0]


@pytest.mark.parametrize("a", ["fp4", "fp8"])
def test_product_bad_counts_are_clamped(G, a):
    import torch
    rng = np.random.default_rng(6)
    N, K, M_cap = 64, 96, 30
    ops = _operands(rng, M_cap, K, 3, N, a)
    for counts, eff, st in (([-5, 10, 4], [0, 10, 4], 1), ([20, 20, 20], [20, 10, 0], 2),
                            ([1 << 30, 1 << 30, 1 << 30], [30, 0, 0], 2)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        offs = torch.full((4,), -7, dtype=torch.int32, device="cuda")
        got = _product(G, counts, M_cap, K, N, a, ops, status, offs)
        assert int(status) == st
        assert offs.tolist() == [0] + np.cumsum(eff).tolist()
        _check(got, eff, sum(eff), ops[4], ops[5], a)


@pytest.mark.parametrize("E,M_cap,N,K", [(70, 30, 64, 96), (3, 2000, 576, 1056)])   # many groups; the 256 x 256 tiles
@pytest.mark.parametrize("a", ["fp4", "fp8"])
def test_product_status_of_every_kernel(G, a, E, M_cap, N, K):
    import torch
    rng = np.random.default_rng(16)
    ops = _operands(rng, M_cap, K, E, N, a)
    half, rest = M_cap // 2, [0] * (E - 3)
    for counts, eff, st in (([half, 5, 0], [half, 5, 0], 0), ([half, -5, 4], [half, 0, 4], 1),
                            ([half, M_cap, 7], [half, M_cap - half, 0], 2),
                            ([-1, M_cap + 1, 7], [0, M_cap, 0], 3), ([1 << 30, 1 << 30, 1 << 30], [M_cap, 0, 0], 2)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        offs = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
        got = _product(G, rest + counts, M_cap, K, N, a, ops, status, offs)
        assert int(status) == st
        assert offs.tolist() == [0] + np.cumsum(rest + eff).tolist()
        _check(got, rest + eff, sum(eff), ops[4], ops[5], a)


@pytest.mark.parametrize("a", ["fp4", "fp8"])
def test_product_many_experts_and_margin(G, a):
    """1024 experts, most of them empty; fewer compute units; the same bits."""
    rng = np.random.default_rng(7)
    counts = np.zeros(1024, np.int64)
    counts[rng.choice(1024, 40, replace=False)] = rng.integers(1, 9, 40)
    M, N, K = int(counts.sum()), 64, 64
    ops = _operands(rng, M, K, 1024, N, a)
    one = _product(G, counts, M, K, N, a, ops)
    _check(one, counts, M, ops[4], ops[5], a)
    assert np.array_equal(one, _product(G, counts, M, K, N, a, ops, cu_margin=250))
    assert np.array_equal(one, _product(G, counts, M, K, N, a, ops))


@pytest.mark.parametrize("a", ["fp4", "fp8"])
def test_product_rows_do_not_depend_on_their_company(G, a):
    """A row's result is the same in bits whatever its neighbours hold and wherever it sits in a group (the same
    capacity, so the same kernel)."""
    rng = np.random.default_rng(8)
    N, K = 128, 736
    for M in (40, 3000):
        ops = _operands(rng, M, K, 1, N, a)
        many = _product(G, [M], M, K, N, a, ops)
        turned = _product(G, [M], M, K, N, a, (np.roll(ops[0], 7, 0), np.roll(ops[1], 7, 0), ops[2], ops[3]))
        assert np.array_equal(np.roll(turned[:M], -7, 0), many[:M])


# groups large enough for the 256 x 256 tiles: whole and short last m-tiles (more and less than 128 rows), N that
# ends inside a tile, K that ends inside a K-tile and in odd numbers of them, empty groups, one row, rows behind
TILE_CASES = [([2000], 576, 1056, 0), ([700, 0, 1, 900, 129], 640, 2880, 7), ([256, 512, 128, 384], 1024, 768, 0),
              ([1300, 1301], 320, 1312, 3), ([255, 257, 511, 1000], 704, 256, 0), ([3000, 5], 256, 7168, 1)]


@pytest.mark.parametrize("a", ["fp4", "fp8"])
@pytest.mark.parametrize("counts,N,K,pad", TILE_CASES)
def test_product_tiles(G, counts, N, K, pad, a):
    rng = np.random.default_rng(N + K + sum(counts))
    M = sum(counts)
    ops = _operands(rng, M + pad, K, len(counts), N, a)
    one = _product(G, counts, M + pad, K, N, a, ops, scale_shift=K % 3)
    _check(one, counts, M, ops[4], ops[5], a)
    # six compute units: several tiles for each workgroup, one stream of K-tiles over them
    few = _product(G, counts, M + pad, K, N, a, ops, cu_margin=250)
    _check(few, counts, M, ops[4], ops[5], a, "six units")


@pytest.mark.parametrize("a", ["fp4", "fp8"])
@pytest.mark.parametrize("counts,N,K", [([1500, 1001], 2048, 32), ([1500, 0, 1001], 2048, 64), ([1301, 3], 2048, 96),
                                        ([2049], 1024, 160), ([2500], 4096, 128), ([700, 1000], 2048, 224),
                                        ([1025, 512], 1024, 352), ([1100], 1024, 480)])
def test_product_short_rows(G, counts, N, K, a):
    """Many rows of fewer blocks than a round of K-tiles: the scales' loads run
    over the rows' ends, and at the arrays' ends are shifted."""
    rng = np.random.default_rng(N + K)
    M = sum(counts)
    ops = _operands(rng, M, K, len(counts), N, a)
    for margin in (0, 250):                     # with few units the tiles are taken from fewer rows on
        got = _product(G, counts, M, K, N, a, ops, cu_margin=margin, scale_shift=K % 3)
        _check(got, counts, M, ops[4], ops[5], a, f"margin {margin}")


@pytest.mark.parametrize("a", ["fp4", "fp8"])
def test_product_tiles_nan_rows_and_columns_stay_their_own(G, a):
    """A NaN scale reaches its row, or its column in its group, and nothing else, across the tiles' edges and
    in rows and columns that share a staged tile."""
    rng = np.random.default_rng(9)
    counts, N, K = [1500, 700], 576, 1056
    M = sum(counts)
    ops = list(_operands(rng, M, K, 2, N, a))
    ops[1][[0, 255, 256, 1499, 1500, M - 1], [0, 5, 32, 7, 31, 32]] = 255
    ops[3][0, [0, 575], [32, 3]] = 255
    got = F.bf16_bits_to_f64(_product(G, counts, M, K, N, a, ops)[:M])
    want = np.zeros((M, N), bool)
    want[[0, 255, 256, 1499, 1500, M - 1]] = True
    want[:1500, [0, 575]] = True
    assert np.array_equal(np.isnan(got), want)


@pytest.mark.parametrize("a", ["fp4", "fp8"])
@pytest.mark.parametrize("E,counts,N,K", [(100, {3: 1, 99: 1}, 64, 32), (65, {0: 17, 64: 3}, 64, 32),
                                          (64, {63: 40}, 64, 32), (1024, {500: 33}, 64, 32),
                                          (100, {3: 1, 99: 1}, 192, 544), (65, {0: 17, 64: 3}, 192, 544),
                                          (64, {63: 40}, 192, 544), (2, {1: 9}, 320, 2080)])
def test_product_few_rows_of_many_experts(G, E, counts, N, K, a):
    rng = np.random.default_rng(E + N)
    c = np.zeros(E, np.int64)
    for e, n in counts.items():
        c[e] = n
    M = int(c.sum())
    ops = _operands(rng, M + 2, K, E, N, a)
    _check(_product(G, c, M + 2, K, N, a, ops, scale_shift=1), c, M, ops[4], ops[5], a)
