"""Residual addition + RMS norm and its gradients on the GPU against the
float64 oracle.

Tolerances, u = 2^-24.  h is equal.  A row sum of H terms at least 64 lanes
wide is off by (H / 64 + 16) u of the sum of the terms' sizes; rstd, half of
that and a root and a quotient: (H / 64 + 24) u of the value; y, three more
products and half a bf16 step.  dx: the same error on each term of the formula
and half a bf16 step; dweight: a sum over T rows in at most 512 shares, each
serial, then the shares: (T / 512 + 512 + 32 + H / 64) u of the sum of the
sizes.  The MXFP8 copy is byte for byte that of moe_mxfp8_quantize."""
import numpy as np
import pytest

import workloads as W
from oracle import formats as F
from oracle import operators as P
from tests.gpu_util import BF16_NAN_SENTINEL, dev_bits, empty_bits, empty_bytes, host_bits

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


SIZES = [(0, 64), (1, 8), (1, 7168), (3, 2880), (2, 2056), (9, 32), (5, 4096), (2, 4128), (2, 8192), (2, 8224),
         (1, 16384), (300, 96), (1, 10000)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("with_res", [True, False])
def test_add_rmsnorm(G, T, H, with_res):
    import torch
    rng = np.random.default_rng(T + H)
    Tb = max(T, 1)
    x, res, wt = _bits(rng, Tb, H), _bits(rng, Tb, H, std=3.0), _bits(rng, H)
    res = res if with_res else None
    h, y, rstd = empty_bits((T + 1, H)), empty_bits((T + 1, H)), torch.full((T + 1,), -7.0, device="cuda")
    mx = q = None
    if H % 32 == 0:
        q, s = empty_bytes((T + 1, H)), empty_bytes((T + 1, H // 32))
        mx = G.mx_out(row_q=q, row_s=s)
    G.moe_add_rmsnorm(dev_bits(x), dev_bits(wt), T, H, 1e-5, residual=None if res is None else dev_bits(res), h=h,
                      y=y, rstd=rstd, mx=mx)
    torch.cuda.synchronize()
    hh, yh, rh = host_bits(h), host_bits(y), rstd.cpu().numpy()
    assert np.all(hh[T] == BF16_NAN_SENTINEL) and np.all(yh[T] == BF16_NAN_SENTINEL) and rh[T] == -7
    if T == 0:
        return
    rhb, rr, ry = P.add_rmsnorm(x, wt, 1e-5, res)
    assert np.array_equal(hh[:T], rhb)
    assert np.all(np.abs(rh[:T] - rr) <= (H / 64 + 24) * U * rr)
    err = np.abs(F.bf16_bits_to_f64(yh[:T]) - ry)
    assert np.all(err <= (2.0 ** -8 + (H / 64 + 32) * U) * np.abs(ry) + 1e-38)
    if q is None:
        return
    q2, s2 = empty_bytes((T + 1, H)), empty_bytes((T + 1, H // 32))
    G.moe_mxfp8_quantize(y, T, H, None, G.mx_out(row_q=q2, row_s=s2))
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("e5m2", [False, True])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_add_rmsnorm_mx_special_rows(G, e5m2, shift):
    """Zero rows, NaN and infinities, the type's extremes, uneven blocks, and
    code buffers of any alignment: the copy is the quantiser's of y."""
    import torch
    rng = np.random.default_rng(11)
    T, H = 8, 160
    v = rng.standard_normal((T, H)) * np.exp2(rng.integers(-12, 12, (T, H // 32))).repeat(32, 1)
    x = W.to_bf16_bits(v.astype(np.float32))
    x[1] = 0
    x[2, 7] = 0x7FC0
    x[3, 70] = 0x7F80
    x[4] = 0x0001                       # the smallest subnormal
    x[5] = 0x7F7F                       # the largest value: its square overflows, rstd is 0
    x[6, 32:] = 0
    wt = _bits(rng, H)
    y = empty_bits((T, H))

    def view(n):
        return empty_bytes((n + 16,))[shift:shift + n]
    q, s, q2, s2 = view(T * H), view(T * H // 32), view(T * H), view(T * H // 32)
    G.moe_add_rmsnorm(dev_bits(x), dev_bits(wt), T, H, 0.0, y=y, mx=G.mx_out(row_q=q, row_s=s, e5m2=e5m2))
    G.moe_mxfp8_quantize(y, T, H, None, G.mx_out(row_q=q2, row_s=s2, e5m2=e5m2))
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2)
    # the copy alone, without y
    q3, s3 = view(T * H), view(T * H // 32)
    G.moe_add_rmsnorm(dev_bits(x), dev_bits(wt), T, H, 0.0, mx=G.mx_out(row_q=q3, row_s=s3, e5m2=e5m2))
    torch.cuda.synchronize()
    assert torch.equal(q3, q2) and torch.equal(s3, s2)


def test_add_rmsnorm_over_its_inputs(G):
    import torch
    rng = np.random.default_rng(12)
    T, H = 7, 2880
    x, res, wt = _bits(rng, T, H), _bits(rng, T, H), _bits(rng, H)
    rhb, _, _ = P.add_rmsnorm(x, wt, 1e-6, res)
    y = []
    for over in (0, 1, None):
        dx, dr = dev_bits(x), dev_bits(res)
        h = empty_bits((T, H)) if over is None else (dx, dr)[over]
        y.append(empty_bits((T, H)))
        G.moe_add_rmsnorm(dx, dev_bits(wt), T, H, 1e-6, residual=dr, h=h, y=y[-1])
        torch.cuda.synchronize()
        assert np.array_equal(host_bits(h), rhb)
    assert torch.equal(y[0], y[2]) and torch.equal(y[1], y[2])


@pytest.mark.parametrize("T,H", [(1, 8), (1, 7168), (3, 2880), (2, 2056), (700, 96), (5, 4096), (2, 8224), (1, 16384),
                                 (2051, 256)])
@pytest.mark.parametrize("with_dh", [True, False])
def test_add_rmsnorm_bwd(G, T, H, with_dh):
    import torch
    rng = np.random.default_rng(T + H + 1)
    h, dy, dh, wt = _bits(rng, T, H, std=2.0), _bits(rng, T, H, std=0.1), _bits(rng, T, H, std=0.1), _bits(rng, H)
    dh = dh if with_dh else None
    rstd = torch.empty(T, device="cuda")
    hd, wd = dev_bits(h), dev_bits(wt)
    G.moe_add_rmsnorm(hd, wd, T, H, 1e-5, rstd=rstd)
    nb = G.moe_add_rmsnorm_bwd_workspace_bytes(T, H)
    ws = torch.full((nb // 4 + 4,), float("nan"), device="cuda")
    dx, dwt = empty_bits((T + 1, H)), torch.full((H + 1,), 3.0, device="cuda")
    dhd = None if dh is None else dev_bits(dh)
    G.moe_add_rmsnorm_bwd(dev_bits(dy), hd, wd, rstd, T, H, dh=dhd, dx=dx, dweight=dwt, workspace=ws)
    torch.cuda.synchronize()
    rdx, rdw = P.add_rmsnorm_bwd(dy, h, wt, 1e-5, dh)
    dyv, hv, wv = (np.abs(F.bf16_bits_to_f64(v)) for v in (dy, h, wt))
    r = 1 / np.sqrt(np.mean(hv * hv, axis=1, keepdims=True) + 1e-5)
    n, g = hv * r, dyv * wv
    mag = r * (g + n * np.mean(g * n, axis=1, keepdims=True)) + (0 if dh is None else np.abs(F.bf16_bits_to_f64(dh)))
    got = host_bits(dx)
    assert np.all(got[T] == BF16_NAN_SENTINEL)
    err = np.abs(F.bf16_bits_to_f64(got[:T]) - rdx)
    assert np.all(err <= 2.0 ** -8 * np.abs(rdx) + 3 * (H / 64 + 32) * U * mag + 1e-38)
    gw = dwt.cpu().numpy()
    assert gw[H] == 3.0 and torch.all(torch.isnan(ws[nb // 4:]))
    dmag = np.sum(dyv * n, axis=0)
    tol = (T / 512 + 512 + 32 + H / 64) * U * dmag + 1e-38
    assert np.all(np.abs(gw[:H] - rdw) <= tol)
    # added to; alone; dx over dh; the same bits again
    dw2 = torch.full((H,), 3.0, device="cuda")
    G.moe_add_rmsnorm_bwd(dev_bits(dy), hd, wd, rstd, T, H, dweight=dw2, accumulate=True, workspace=ws)
    over = None if dh is None else dev_bits(dh)
    dx2 = empty_bits((T, H)) if over is None else over
    G.moe_add_rmsnorm_bwd(dev_bits(dy), hd, wd, rstd, T, H, dh=over, dx=dx2)
    dw3 = torch.zeros(H, device="cuda")
    G.moe_add_rmsnorm_bwd(dev_bits(dy), hd, wd, rstd, T, H, dweight=dw3, workspace=ws)
    torch.cuda.synchronize()
    assert np.all(np.abs(dw2.cpu().numpy() - 3 - rdw) <= tol + 4 * U * (3 + np.abs(rdw)))
    assert torch.equal(dx2, dx[:T]) and torch.equal(dw3, dwt[:H])


def test_add_rmsnorm_zeros_keep_their_sign(G):
    import torch
    rng = np.random.default_rng(8)
    x, wt = _bits(rng, 5, 256), _bits(rng, 256)
    x[:, ::3] = 0x0000
    x[:, 1::3] = 0x8000
    x[4] = 0x8000                                     # a row of zeros alone
    y = empty_bits((5, 256))
    G.moe_add_rmsnorm(dev_bits(x), dev_bits(wt), 5, 256, 1e-5, y=y)
    torch.cuda.synchronize()
    got = host_bits(y)
    zero = (x & 0x7FFF) == 0
    assert np.array_equal(got[zero], ((x ^ wt) & 0x8000)[zero]) and np.all((got & 0x7FFF)[~zero] != 0)


def test_add_rmsnorm_rounds_once(G):
    """y is rounded to fp32 and then to bf16, from a product kept in two floats."""
    import torch
    rng = np.random.default_rng(9)
    T, H = 96, 7168
    x, wt = _bits(rng, T, H), _bits(rng, H)
    y = empty_bits((T, H))
    G.moe_add_rmsnorm(dev_bits(x), dev_bits(wt), T, H, 2.0 ** -20, y=y)
    torch.cuda.synchronize()
    _, _, want = P.add_rmsnorm(x, wt, 2.0 ** -20)
    got = F.bf16_bits_to_f64(host_bits(y))
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -126))) - 7)
    # half a step of bf16, and half a step of fp32 (2^-17 of it), half as much again for the parts left out
    assert np.all(np.abs(got - want) <= step * (0.5 + 1.5 * 2.0 ** -17))


def test_add_rmsnorm_bwd_no_rows(G):
    import torch
    one = empty_bits((1, 64))
    dwt = torch.full((64,), 3.0, device="cuda")
    rstd = torch.ones(1, device="cuda")
    G.moe_add_rmsnorm_bwd(one, one, one, rstd, 0, 64, dweight=dwt)
    torch.cuda.synchronize()
    assert torch.all(dwt == 0)
    G.moe_add_rmsnorm_bwd(one, one, one, rstd, 0, 64, dweight=dwt.fill_(2.0), accumulate=True)
    torch.cuda.synchronize()
    assert torch.all(dwt == 2.0)


def test_add_rmsnorm_gradient_against_differences(G):
    """dx against central differences of L = <dy, y> in float64 from the
    oracle's forward (its own rounding left out): step 2^-10, error h^2 / 6
    |L'''| with |L'''| <= 30 sum |dy w| / H^(1/2), and the kernel's half bf16 step."""
    import torch
    rng = np.random.default_rng(13)
    H, e = 16, 2.0 ** -10
    h, dy, wt = _bits(rng, 1, H), _bits(rng, 1, H), _bits(rng, H)
    hv, dyv, wv = (F.bf16_bits_to_f64(v) for v in (h, dy, wt))

    def loss(a):
        return np.sum(dyv * a / np.sqrt(np.mean(a * a) + 1e-5) * wv)
    num = np.array([(loss(hv + e * np.eye(H)[i]) - loss(hv - e * np.eye(H)[i])) / (2 * e) for i in range(H)])
    rstd, dx = torch.empty(1, device="cuda"), empty_bits((1, H))
    G.moe_add_rmsnorm(dev_bits(h), dev_bits(wt), 1, H, 1e-5, rstd=rstd)
    G.moe_add_rmsnorm_bwd(dev_bits(dy), dev_bits(h), dev_bits(wt), rstd, 1, H, dx=dx)
    torch.cuda.synchronize()
    got = F.bf16_bits_to_f64(host_bits(dx))[0]
    tol = e * e / 6 * 30 * np.sum(np.abs(dyv * wv)) + 2.0 ** -8 * np.abs(num) + 1e-5
    assert np.all(np.abs(got - num) <= tol)
