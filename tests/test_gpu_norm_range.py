"""The norm of rows whose squares fp32 does not hold: too large (bf16 reaches
3.4e38, whose square is 1e77), or, with a small eps, too small.

Tolerances, u = 2^-24, as in test_gpu_norm: rstd is one rounding of a value in
64 bits, or half a step of its subnormals (2^-150), and inf where it passes
fp32's range; y half a bf16 step and three roundings, and half a step of bf16's
subnormals (2^-134); dx as there, with rstd's relative error as one more."""
import numpy as np
import pytest

import workloads as W
from oracle import formats as F
from oracle import operators as P
from tests.gpu_util import dev_bits, empty_bits, host_bits
from tests.test_gpu_norm import G, U  # noqa: F401  (G: the fixture)

pytestmark = pytest.mark.gpu
POWERS = [-133, -130, -126, -100, -64, -63, -62, -50, -20, 0, 40, 62, 63, 64, 100, 125]


def _rows(rng, H):
    """A row of values around 2^p for each p (at most 3 2^p in size)."""
    v = np.clip(rng.standard_normal((len(POWERS), H)), -3, 3)
    v = np.where(np.arange(H) % 7 == 3, 0.0, v)
    bits = W.to_bf16_bits((v * np.exp2(np.array(POWERS, float))[:, None]).astype(np.float32))
    return bits


@pytest.mark.parametrize("repeat", [1, 40])             # a workgroup of 1024 threads for few rows, of 256 for many
@pytest.mark.parametrize("H", [8, 256, 7168, 16384])
@pytest.mark.parametrize("eps", [0.0, 1e-36, 1e-5])
def test_norm_of_large_and_small_rows(G, H, eps, repeat):  # noqa: F811
    import torch
    rng = np.random.default_rng(H)
    x = np.concatenate([_rows(rng, H)] * repeat)
    T = len(x)
    wt = W.to_bf16_bits(rng.standard_normal(H).astype(np.float32))
    eps = float(np.float32(eps))
    y, h, rstd = empty_bits((T, H)), empty_bits((T, H)), torch.empty(T, device="cuda")
    G.moe_add_rmsnorm(dev_bits(x), dev_bits(wt), T, H, eps, h=h, y=y, rstd=rstd)
    torch.cuda.synchronize()
    n = len(POWERS)
    hb, rs, yv = P.add_rmsnorm(x[:n], wt, eps)
    yh, got = host_bits(y), rstd.double().cpu().numpy()
    assert np.all(yh.reshape(repeat, n, H) == yh[:n]) and np.array_equal(host_bits(h)[:n], hb)
    inf = rs >= 2.0 ** 128 * (1 - U / 2)
    assert np.all(np.isinf(got[:n][inf])) and np.all(np.isfinite(got[:n][~inf]))
    assert np.all(np.abs(got[:n] - rs)[~inf] <= 4 * U * rs[~inf] + 2.0 ** -150)
    err = np.abs(F.bf16_bits_to_f64(yh[:n]) - yv)
    assert np.all(err <= (2.0 ** -8 + 4 * U) * np.abs(yv) + 2.0 ** -134)


def test_norm_of_large_sums_with_the_residual(G):  # noqa: F811
    rng = np.random.default_rng(2)
    H = 2880
    x, res, wt = _rows(rng, H), _rows(rng, H), W.to_bf16_bits(rng.standard_normal(H).astype(np.float32))
    y, h = empty_bits(x.shape), empty_bits(x.shape)
    G.moe_add_rmsnorm(dev_bits(x), dev_bits(wt), len(x), H, 0.0, residual=dev_bits(res), h=h, y=y)
    hb, _, yv = P.add_rmsnorm(x, wt, 0.0, res)
    assert np.array_equal(host_bits(h), hb)
    err = np.abs(F.bf16_bits_to_f64(host_bits(y)) - yv)
    assert np.all(err <= (2.0 ** -8 + 4 * U) * np.abs(yv) + 2.0 ** -134)


def test_norm_of_infinite_and_nan_rows_stays(G):  # noqa: F811
    """mean = inf: rstd 0, the infinities themselves NaN; a NaN takes its row; a row of zeros without eps is NaN."""
    import torch
    H = 64
    x = W.to_bf16_bits(np.random.default_rng(3).standard_normal((4, H)).astype(np.float32))
    x[0, 5], x[1, 6], x[2] = 0x7F80, 0x7FC0, 0
    wt = W.to_bf16_bits(np.ones(H, np.float32))
    y, rstd = empty_bits((4, H)), torch.empty(4, device="cuda")
    G.moe_add_rmsnorm(dev_bits(x), dev_bits(wt), 4, H, 0.0, y=y, rstd=rstd)
    got, r = F.bf16_bits_to_f64(host_bits(y)), rstd.cpu().numpy()
    assert r[0] == 0 and np.isnan(got[0, 5]) and np.all(np.delete(got[0], 5) == 0)
    assert np.isnan(r[1]) and np.all(np.isnan(got[1])) and np.isinf(r[2]) and np.all(np.isnan(got[2]))
    assert np.all(np.isfinite(got[3]))


def test_norm_gradients_of_large_rows(G):  # noqa: F811
    import torch
    rng = np.random.default_rng(4)
    H = 512
    keep = [i for i, p in enumerate(POWERS) if -64 <= p <= 100]
    h, T = _rows(rng, H)[keep], len(keep)
    wt, dy = (W.to_bf16_bits(rng.standard_normal(s).astype(np.float32)) for s in ((H,), (T, H)))
    rstd, dx, dw = torch.empty(T, device="cuda"), empty_bits((T, H)), torch.empty(H, device="cuda")
    ws = torch.empty(G.moe_add_rmsnorm_bwd_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    hd, wd = dev_bits(h), dev_bits(wt)
    G.moe_add_rmsnorm(hd, wd, T, H, 0.0, rstd=rstd)
    G.moe_add_rmsnorm_bwd(dev_bits(dy), hd, wd, rstd, T, H, dx=dx, dweight=dw, workspace=ws)
    torch.cuda.synchronize()
    rdx, rdw = P.add_rmsnorm_bwd(dy, h, wt, 0.0)
    dyv, hv, wv = (np.abs(F.bf16_bits_to_f64(v)) for v in (dy, h, wt))
    r = 1 / np.sqrt(np.mean(hv * hv, axis=1, keepdims=True))
    n, g = hv * r, dyv * wv
    mag = r * (g + n * np.mean(g * n, axis=1, keepdims=True))
    err = np.abs(F.bf16_bits_to_f64(host_bits(dx)) - rdx)
    assert np.all(err <= 2.0 ** -8 * np.abs(rdx) + 3 * (H / 64 + 32) * U * mag + 1e-38)
    dmag = np.sum(dyv * n, axis=0)
    assert np.all(np.abs(dw.cpu().numpy() - rdw) <= (T / 512 + 512 + 32 + H / 64) * U * dmag + 1e-38)
