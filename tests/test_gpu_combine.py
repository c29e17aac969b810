"""The combine and its gradients on the GPU against the float64 oracle.

Tolerances, u = 2^-24: an output of k products and k additions in fp32 is off
by at most (k + 2) u times the sum of the terms' sizes, then half a bf16 step
(2^-8 of the value); a dot product of H terms, at least 64 lanes wide, by
(H / 64 + 16) u times the sum of the products' sizes; dy is one product and
one rounding to bf16."""
import numpy as np
import pytest

import workloads as W
from oracle import formats as F
from oracle import operators as P
from tests.gpu_util import BF16_NAN_SENTINEL, dev_bits, empty_bits, host_bits

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


def _bits(rng, *shape, std=1.0):
    return W.to_bf16_bits((rng.standard_normal(shape) * std).astype(np.float32))


def _dst(rng, T, k, M, drop):
    d = rng.permutation(M)[:T * k].reshape(T, k).astype(np.int32)
    d[rng.random((T, k)) < drop] = -1
    return d


def _forward(G, y, dst, w, res, inplace=False):
    import torch
    M, H = y.shape
    T, k = dst.shape
    out = empty_bits((T + 1, H))
    dres = None if res is None else dev_bits(res)
    if inplace:
        out[:T] = dres
        dres = out
    dd = torch.from_numpy(dst).cuda() if T else torch.zeros(1, k, dtype=torch.int32, device="cuda")
    G.moe_combine(dev_bits(y), M, H, dd, T, k, out, weights=None if w is None else torch.from_numpy(w).cuda(),
                  residual=dres)
    torch.cuda.synchronize()
    got = host_bits(out)
    assert np.all(got[T] == BF16_NAN_SENTINEL)
    want = P.combine(y, dst, w, res)
    mag = P.combine(y & 0x7FFF, dst, None if w is None else np.abs(w), None if res is None else res & 0x7FFF)
    err = np.abs(F.bf16_bits_to_f64(got[:T]) - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + (k + 2) * U * 1.01 * mag + 1e-37)


@pytest.mark.parametrize("T,k,H", [(0, 2, 64), (1, 1, 8), (1, 8, 7168), (3, 4, 2880), (17, 16, 24), (5, 3, 2056),
                                   (200, 8, 512), (64, 6, 4104)])
@pytest.mark.parametrize("with_w,with_res", [(True, True), (True, False), (False, False)])
def test_combine(G, T, k, H, with_w, with_res):
    rng = np.random.default_rng(T + k + H)
    M = T * k + 5
    y = _bits(rng, M, H)
    w = rng.random((T, k)).astype(np.float32) - 0.25 if with_w else None
    res = _bits(rng, T, H, std=3.0) if with_res else None
    _forward(G, y, _dst(rng, T, k, M, 0.2), w if T else None, res if T else None)


def test_combine_rows_left_out_and_repeated(G):
    """No row for a token, rows beyond the capacity, one row in two slots and
    in two tokens; NaN in rows that no pair names changes nothing; the output
    over the residual."""
    rng = np.random.default_rng(1)
    M, H = 9, 72
    y = _bits(rng, M, H)
    y[8] = BF16_NAN_SENTINEL
    dst = np.array([[-1, -1, -1], [9, 1 << 30, -(1 << 31)], [2, 2, 5], [2, 7, -5], [0, 1, 3]], dtype=np.int32)
    w = rng.standard_normal((5, 3)).astype(np.float32)
    w[0] = np.nan                     # of pairs without a row
    res = _bits(rng, 5, H)
    _forward(G, y, dst, w, res)
    _forward(G, y, dst, w, None)
    _forward(G, y, dst, w, res, inplace=True)


def _backward(G, dout, y, dst, w, want_dy=True, want_dw=True):
    import torch
    M, H = y.shape
    T, k = dst.shape
    dy = empty_bits((M, H)) if want_dy else None
    dw = torch.full((T + 1, k), -7.0, device="cuda") if want_dw else None
    G.moe_combine_bwd(dev_bits(dout), dev_bits(y) if want_dw else None, M, H, torch.from_numpy(dst).cuda(), T, k,
                      weights=None if w is None else torch.from_numpy(w).cuda(), dy=dy, dweights=dw)
    torch.cuda.synchronize()
    rdy, named, rdw = P.combine_bwd(dout, y, dst, w)
    if want_dy:
        got = host_bits(dy)
        assert np.all(got[~named] == BF16_NAN_SENTINEL)          # rows that no pair names
        g = F.bf16_bits_to_f64(got[named])
        mag, _, _ = P.combine_bwd(dout & 0x7FFF, y, dst, None if w is None else np.abs(w))
        assert np.all(np.abs(g - rdy[named]) <= 2.0 ** -8 * np.abs(rdy[named]) + 3 * U * mag[named] + 1e-37)
    if want_dw:
        got = dw.cpu().numpy()
        assert np.all(got[T] == -7)
        _, _, mag = P.combine_bwd(dout & 0x7FFF, y & 0x7FFF, dst, w)
        assert np.all(np.abs(got[:T] - rdw) <= (H / 64 + 16) * U * mag + 1e-37)
        assert np.all(got[:T][(dst < 0) | (dst >= M)] == 0)


@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (1, 8, 7168), (3, 4, 2880), (17, 16, 24), (5, 3, 2056), (200, 8, 512),
                                   (64, 6, 4104)])
def test_combine_bwd(G, T, k, H):
    rng = np.random.default_rng(T + k + H + 1)
    M = T * k + 5
    y, dout = _bits(rng, M, H), _bits(rng, T, H, std=0.1)
    w = rng.random((T, k)).astype(np.float32)
    dst = _dst(rng, T, k, M, 0.2)
    _backward(G, dout, y, dst, w)
    _backward(G, dout, y, dst, None)
    _backward(G, dout, y, dst, w, want_dw=False)
    _backward(G, dout, y, dst, w, want_dy=False)


def test_combine_bwd_repeated_row_of_one_token(G):
    rng = np.random.default_rng(2)
    y, dout = _bits(rng, 8, 40), _bits(rng, 3, 40)
    dst = np.array([[2, 2, 2, 5], [-1, -1, -1, -1], [7, 0, 7, 9]], dtype=np.int32)
    _backward(G, dout, y, dst, rng.standard_normal((3, 4)).astype(np.float32))


def test_combine_gradient_against_differences(G):
    """L = <dout, out> is linear in the weights: on values that stay exact in
    bf16 and fp32 (small integers), the difference of two forward passes is the
    gradient to the bit."""
    import torch
    rng = np.random.default_rng(3)
    T, k, H, M = 4, 3, 16, 12
    y = W.to_bf16_bits(rng.integers(-2, 3, (M, H)).astype(np.float32))
    dout = W.to_bf16_bits(rng.integers(-2, 3, (T, H)).astype(np.float32))
    dst = _dst(rng, T, k, M, 0.0)
    w = rng.integers(-2, 3, (T, k)).astype(np.float32)
    dd, yd, dwt = torch.from_numpy(dst).cuda(), dev_bits(y), torch.empty(T, k, device="cuda")
    G.moe_combine_bwd(dev_bits(dout), yd, M, H, dd, T, k, weights=torch.from_numpy(w).cuda(), dweights=dwt)

    def loss(wh):
        out = empty_bits((T, H))
        G.moe_combine(yd, M, H, dd, T, k, out, weights=torch.from_numpy(wh).cuda())
        torch.cuda.synchronize()
        return np.sum(F.bf16_bits_to_f64(host_bits(out)) * F.bf16_bits_to_f64(dout))
    base = loss(w)
    got = dwt.cpu().numpy()
    for t in range(T):
        for j in range(k):
            w2 = w.copy()
            w2[t, j] += 1
            assert loss(w2) - base == got[t, j]


def test_combine_is_the_gradient_of_the_row_gather(G):
    """With no weights: dx = the sum of a token's gathered rows' gradients."""
    rng = np.random.default_rng(4)
    dst = _dst(rng, 50, 4, 200, 0.0)
    _forward(G, _bits(rng, 200, 128), dst, None, None)
