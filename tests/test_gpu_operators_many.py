"""More tokens than a launch has workgroups, the most tokens that the router
takes, and the widest rows that the combine takes.  On small integers, whose
sums are exact, or sampled against the float64 oracle with the operators' own
tolerances."""
import numpy as np
import pytest

from oracle import formats as F
from oracle import operators as P
from tests.gpu_util import host_bits
from tests.test_gpu_router import G, U  # noqa: F401  (G: the fixture)

pytestmark = pytest.mark.gpu


def _ints(g, *shape):
    import torch
    return torch.randint(-3, 4, shape, generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)


@pytest.mark.parametrize("T,k,H", [((1 << 20) + 37, 2, 8), (3 * (1 << 20) + 1, 1, 16), (2, 1, 1 << 26), (1, 3, (1 << 25) + 8)])
def test_combine_and_gradients(G, T, k, H):  # noqa: F811
    """Every row named once, by the pairs in another order; a few pairs dropped."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    M = T * k
    y, dout, res = _ints(g, M, H), _ints(g, T, H), _ints(g, T, H)
    dst = torch.randperm(M, generator=g, device="cuda").int().view(T, k)
    if T > 100:
        dst[torch.rand(T, k, generator=g, device="cuda") < 0.01] = -1
    w = torch.randint(-2, 3, (T, k), generator=g, device="cuda").float()
    out = torch.empty_like(res)
    G.moe_combine(y, M, H, dst, T, k, out, weights=w, residual=res)
    want = res.float()
    at = dst.clamp(min=0).long()
    there = (dst >= 0).float()
    for j in range(k):
        want += y[at[:, j]].float() * (w[:, j] * there[:, j])[:, None]
    assert torch.equal(out, want.to(torch.bfloat16))
    del want, out, res
    dy, dw = torch.full_like(y, 7.0), torch.full((T, k), 7.0, device="cuda")
    G.moe_combine_bwd(dout, y, M, H, dst, T, k, weights=w, dy=dy, dweights=dw)
    for j in range(k):
        sel = dst[:, j] >= 0
        rows = at[sel, j]
        want = (dout[sel].float() * w[sel, j][:, None]).to(torch.bfloat16)
        assert torch.equal(dy[rows], want)
        dot = (dout[sel].double() * y[rows].double()).sum(1)
        # (sums of integers of at most 9 H: exact in fp32 up to 2^24)
        err = (dw[sel, j].double() - dot).abs()
        assert bool((err <= (0 if 9 * H < 1 << 24 else (H / 64 + 16) * U * 9 * H)).all()) and bool((dw[~sel, j] == 0).all())
    named = torch.zeros(M, dtype=torch.bool, device="cuda")
    named[dst[dst >= 0].long()] = True
    assert bool((dy[~named] == 7).all())


@pytest.mark.parametrize("H", [8, 64])
def test_norm_of_many_rows(G, H):  # noqa: F811
    import torch
    T = (1 << 20) + 41
    g = torch.Generator(device="cuda").manual_seed(H)
    x, res = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    wt = torch.randn(H, generator=g, device="cuda").bfloat16()
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda")
    G.moe_add_rmsnorm(x, wt, T, H, 1e-5, residual=res, h=h, y=y, rstd=rstd)
    assert torch.equal(h, x + res)                          # (torch rounds the fp32 sum once, too)
    f = h.double()
    r = 1 / torch.sqrt((f * f).mean(1, keepdim=True) + float(np.float32(1e-5)))
    want = f * r * wt.double()
    assert bool(((y.double() - want).abs() <= (2.0 ** -8 + 4 * U) * want.abs() + 2.0 ** -134).all())
    assert bool(((rstd.double() - r[:, 0]).abs() <= 4 * U * r[:, 0]).all())
    # the gradients: rows in 512 shares
    dy = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    ws = torch.empty(G.moe_add_rmsnorm_bwd_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    G.moe_add_rmsnorm_bwd(dy, h, wt, rstd, T, H, dx=dx, dweight=dw, workspace=ws)
    n, gw = f * r, dy.double() * wt.double()
    rdx = r * (gw - n * (gw * n).mean(1, keepdim=True))
    mag = r * (gw.abs() + n.abs() * (gw * n).abs().mean(1, keepdim=True))
    assert bool(((dx.double() - rdx).abs() <= 2.0 ** -8 * rdx.abs() + 3 * (H / 64 + 32) * U * mag + 1e-38).all())
    t = dy.double() * n
    assert bool(((dw.double() - t.sum(0)).abs() <= (T / 512 + 512 + 32 + H / 64) * U * t.abs().sum(0)).all())


@pytest.mark.parametrize("E,k", [(4, 2), (5, 1)])          # 16 lanes per token; a wave per token in 64 bits
def test_router_most_tokens(G, E, k):  # noqa: F811
    import torch
    T = 1 << 25
    g = torch.Generator(device="cuda").manual_seed(E)
    x = torch.randn(T, E, generator=g, device="cuda").bfloat16()
    ids, w = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda"), torch.full((T + 1, k), -7.0, device="cuda")
    r = G.router("sigmoid", renorm=True, scale=1.5)
    G.moe_router_topk(x, T, E, k, r, ids, w)
    assert ids[T].tolist() == [-7] * k and w[T].tolist() == [-7.0] * k
    best = x.float().sort(dim=1, descending=True, stable=True).indices[:, :k].int()
    assert torch.equal(ids[:T], best)
    rows = [0, 1, 2, 3, 1 << 23, T // 2 + 5, T - 3, T - 1]
    v = x[rows].double().cpu().numpy()
    rid, rw = P.router_topk(v, k, score="sigmoid", scale=1.5)
    assert np.array_equal(ids[rows].cpu().numpy(), rid)
    assert np.all(np.abs(w[rows].cpu().numpy() - rw) <= (2 * 6 + 32) * U * rw)
    d, dw = torch.full((T + 1, E), 7.0, device="cuda").bfloat16(), torch.ones(T, k, device="cuda")
    dw[:, 0] = -2.0
    G.moe_router_topk_bwd(x, T, E, k, r, ids, dw, d)
    assert bool((d[T] == 7).all())
    want = P.router_topk_bwd(v, rid, dw[rows].cpu().numpy(), "sigmoid", True, 1.5)
    err = np.abs(F.bf16_bits_to_f64(host_bits(d[rows].view(torch.int16))) - want)
    # terms of at most 1.5 x (2 + 2) each
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + 4 * (2 * 6 + 32) * U * 6)
    torch.cuda.empty_cache()
