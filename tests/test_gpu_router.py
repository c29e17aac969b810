"""The router and its gradient on the GPU against the float64 oracle.

Tolerances.  ids are equal.  Weights: with u = 2^-24 and R the largest |logit
- row maximum| (or |logit|), an fp32 exponential is off by at most (2 R + 2) u
(its argument's rounding and the multiplication by log2 e, then the function's
own), a sum of up to 1024 positive terms in 16 per lane and 6 halvings by 22 u,
a quotient by 2 u: (2 R + 32) u of the value covers them.  Gradients: the same
relative error on each term of the formula, on the sum of the terms' sizes
(4 times, for the products of up to three such factors), and half a bf16 step
(2^-8) where the output is bf16."""
import numpy as np
import pytest

import workloads as W
from oracle import formats as F
from oracle import operators as P

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


def _logits(x, bf16):
    """(device logits of at least one row, their float64 values)"""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32))
    if bf16:
        t = t.to(torch.bfloat16)
    v = t.double().numpy()
    if len(x) == 0:
        t = torch.zeros((1,) + tuple(t.shape[1:]), dtype=t.dtype)
    return t.cuda(), v


def _reach(v, score):
    """R of the module's docstring, per row, over the finite logits."""
    with np.errstate(invalid="ignore"):
        f = np.where(np.isfinite(v), v, np.nan)
        if score == "sigmoid":
            r = np.nanmax(np.abs(f), axis=1, initial=0)
        else:
            r = np.nanmax(f, axis=1, initial=-1e4) - np.nanmin(f, axis=1, initial=1e4)
    return np.clip(r, 0, 100)[:, None]


def _run(G, x, k, bf16=False, bias=None, dw=None, **kw):
    import torch
    T, E = x.shape
    lg, v = _logits(x, bf16)
    r = G.router(bias=None if bias is None else torch.from_numpy(bias).cuda(), **kw)
    ids = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    G.moe_router_topk(lg, T, E, k, r, ids, w)
    torch.cuda.synchronize()
    ids_h, w_h = ids.cpu().numpy(), w.cpu().numpy()
    assert np.all(ids_h[T] == -7) and np.all(w_h[T] == -7)          # nothing behind the last token
    okw = {a: b for a, b in kw.items()}
    rid, rw = P.router_topk(v, k, bias=bias, **okw)
    assert np.array_equal(ids_h[:T], rid)
    R = _reach(v, kw.get("score", "softmax"))
    assert np.array_equal(np.isnan(w_h[:T]), np.isnan(rw))
    fin = ~np.isnan(rw)
    tol = np.broadcast_to((2 * R + 32) * U, rw.shape)
    assert np.all(np.abs(w_h[:T] - rw)[fin] <= (tol * np.abs(rw) + 1e-37)[fin])
    if dw is None:
        return
    d = torch.full((T + 1, E), -7.0, device="cuda").to(lg.dtype)
    dwd = torch.zeros(T + 1, k, device="cuda")           # (at least one row, so that T = 0 has a pointer)
    dwd[:T] = torch.from_numpy(np.ascontiguousarray(dw, dtype=np.float32)).cuda()
    G.moe_router_topk_bwd(lg, T, E, k, r, ids, dwd, d)
    torch.cuda.synchronize()
    got = d.double().cpu().numpy()
    assert np.all(got[T] == -7)
    _check_grad(got[:T], v, rid, dw, R, bf16, **kw)


def _check_grad(got, v, ids, dw, R, bf16, score="softmax", renorm=True, scale=1.0, **_):
    dw = np.asarray(dw, dtype=np.float32).astype(np.float64)
    want = P.router_topk_bwd(v, ids, dw, score, renorm, scale)
    # the sizes of the formula's terms
    mag = np.zeros_like(want)
    for t in range(len(v)):
        s = P.router_scores(v[t], score)
        S = s[ids[t]].sum() if renorm else 1.0
        if not S > 0:
            continue
        dot = (np.abs(dw[t]) * s[ids[t]]).sum() / S
        ds = np.zeros(v.shape[1])
        np.add.at(ds, ids[t], abs(scale) / S * (np.abs(dw[t]) + (dot if renorm else 0)))
        mag[t] = s * ds if score == "sigmoid" else s * (ds + (s * ds).sum())
    tol = 4 * (2 * R + 32) * U * mag + (2.0 ** -8 if bf16 else U) * np.abs(want) + 1e-37
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(0, 8, 2), (1, 1, 1), (3, 5, 5), (257, 64, 6), (70, 65, 8), (33, 200, 16),
                                   (19, 256, 8), (9, 513, 3), (6, 1024, 16), (1030, 128, 4), (75, 512, 8),
                                   (21, 36, 16)])
def test_router_sizes(G, T, E, k, score, bf16):
    rng = np.random.default_rng(T + E + k)
    x = rng.standard_normal((T, E)) * 2
    for renorm, scale in ((True, 1.0), (False, 2.5)):
        _run(G, x, k, bf16, None, rng.standard_normal((T, k)), score=score, renorm=renorm, scale=scale)


# more tokens than take a wave each
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score,with_bias,group_score", [("softmax", False, "top2"), ("sigmoid", True, "top2"),
                                                         ("softmax", True, "max"), ("sigmoid", False, "max")])
@pytest.mark.parametrize("T,E,k,groups,keep", [(2049, 68, 5, 1, 1), (2053, 128, 6, 8, 4), (2050, 200, 16, 1, 1),
                                               (2051, 256, 8, 8, 4), (2052, 264, 7, 1, 1), (2049, 512, 10, 4, 2),
                                               (2050, 256, 8, 2, 1)])
def test_router_many_tokens(G, T, E, k, groups, keep, score, with_bias, group_score, bf16):
    rng = np.random.default_rng(T + E)
    bias = (rng.standard_normal(E) * 0.2).astype(np.float32) if with_bias else None
    x = rng.standard_normal((T, E))
    x[7] = -np.inf
    x[8, ::2] = -np.inf
    x[9, 3] = np.nan
    _run(G, x, k, bf16, bias, None, score=score, n_groups=groups, topk_groups=keep, group_score=group_score, scale=1.5)


@pytest.mark.parametrize("score,group_score", [("softmax", "max"), ("softmax", "top2"), ("sigmoid", "max"),
                                               ("sigmoid", "top2")])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,groups,keep", [(61, 256, 8, 8, 4), (40, 160, 6, 8, 3), (33, 512, 10, 4, 2), (30, 12, 3, 4, 1),
                                               (20, 128, 2, 64, 1), (15, 1024, 16, 16, 16), (25, 21, 7, 3, 2)])
def test_router_groups_and_bias(G, T, E, k, groups, keep, with_bias, score, group_score):
    if group_score == "top2" and E // groups < 2:
        pytest.skip("a group of one expert has no second score")
    rng = np.random.default_rng(E + keep)
    bias = (rng.standard_normal(E) * 0.2).astype(np.float32) if with_bias else None
    for bf16 in (False, True):   # bf16 logits hold many exact ties, of groups too
        _run(G, rng.standard_normal((T, E)), k, bf16, bias, rng.standard_normal((T, k)), score=score,
             n_groups=groups, topk_groups=keep, group_score=group_score, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,keep,group_score", [(1, 1, "max"), (4, 2, "max"), (4, 2, "top2")])
def test_router_masks_ties_and_special_values(G, score, groups, keep, group_score):
    inf, nan, low = np.inf, np.nan, np.finfo(np.float32).min
    E = 96
    rng = np.random.default_rng(3)
    x = rng.standard_normal((14, E)).astype(np.float32)
    x[0] = -inf                      # every expert masked
    x[1] = low                       # masked with the type's lowest value
    x[2, 1:] = -inf                  # one expert left
    x[3, ::2] = -inf                 # every other expert masked
    x[4] = 0.5                       # all equal: the lowest ids
    x[5, :48], x[5, 48:] = 0.0, -0.0
    x[6, 5] = nan
    x[7] = nan
    x[8, 7] = inf
    x[9, 3], x[9, 4] = 80.0, -80.0
    x[10, 90:] = low
    x[11] = -200.0                   # sigmoid scores that fp32 cannot hold
    x[12] = np.repeat(rng.standard_normal(E // 8), 8)   # ties inside groups
    x[13, 0] = nan
    x[13, 1:] = -inf
    for renorm in (True, False):
        _run(G, x, 4, False, None, None, score=score, renorm=renorm, n_groups=groups, topk_groups=keep,
             group_score=group_score)
    bias = np.where(np.arange(E) % 5 == 0, 0.25, 0.0).astype(np.float32)
    _run(G, x[[0, 2, 3, 4, 6, 7, 12]], 4, False, bias, None, score=score, n_groups=groups, topk_groups=keep,
         group_score=group_score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_neighbouring_scores(G, score):
    """Logits one unit apart, where fp32 scores would tie or swap: the choice
    follows the formula, with and without a bias and groups."""
    E = 64
    base = np.float32(6.0)
    x = np.empty((8, E), np.float32)
    rng = np.random.default_rng(4)
    for t in range(8):
        v = base
        vals = []
        for _ in range(E):
            vals.append(v)
            v = np.nextafter(v, np.float32(100))
        x[t] = np.array(vals)[rng.permutation(E)]
    _run(G, x, 8, score=score)
    _run(G, x, 8, bias=np.zeros(E, np.float32), score=score)
    _run(G, x, 8, bias=np.full(E, 0.125, np.float32), score=score, n_groups=8, topk_groups=3, group_score="top2")
    _run(G, x, 8, score=score, n_groups=8, topk_groups=3, group_score="top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_router_gradient_masks_foreign_and_repeated_ids(G, score, renorm):
    import torch
    inf = np.inf
    rng = np.random.default_rng(5)
    T, E, k = 6, 10, 4
    x = rng.standard_normal((T, E)).astype(np.float32)
    x[0] = -inf
    x[1, 3:] = -inf
    ids = np.array([[0, 1, 2, 3], [0, 1, 2, 3], [4, 4, 1, 0], [-1, 10, 2, 3], [-1, 11, 1 << 30, -9], [9, 8, 7, 9]],
                   dtype=np.int32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    lg, v = _logits(x, False)
    d = torch.full((T, E), 7.0, device="cuda")
    r = G.router(score, renorm=renorm, scale=1.5)
    G.moe_router_topk_bwd(lg, T, E, k, r, torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), d)
    torch.cuda.synchronize()
    got = d.double().cpu().numpy()
    want = P.router_topk_bwd(v, ids, dw, score, renorm, 1.5)
    assert np.all(got[0] == 0) and np.all(got[4] == 0)
    # sizes: |dw| <= 3, scale 1.5, at most 4 terms each with a factor 1 / S <= 1 / s: bounded by 4 x 1.5 x 3 x 2
    assert np.max(np.abs(got - want)) <= 4 * (2 * 6 + 32) * U * 36


def test_router_gradient_against_differences(G):
    """Central differences of the GPU's own weights in float64 logits would
    need a float64 kernel; with h = 2^-6 in fp32 the difference quotient of L =
    <dw, w> is off by h^2 / 6 |L'''| (|L'''| <= 10 |dw| here) and by 2 x 8 u |L|
    / 2h from the weights' rounding."""
    import torch
    rng = np.random.default_rng(6)
    E, k, h = 12, 3, 2.0 ** -6
    x = np.round(rng.standard_normal(E) * 64) / 64
    dw = rng.standard_normal(k).astype(np.float32)
    for score, renorm in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        r = G.router(score, renorm=renorm)
        ids0 = P.router_topk(x[None], k, score, renorm=renorm)[0]
        rows = np.concatenate([x[None] + h * np.eye(E), x[None] - h * np.eye(E)]).astype(np.float32)
        s = [P.router_scores(v.astype(np.float64), score)[ids0[0]] for v in rows]
        L = np.array([np.sum(dw * (a / a.sum() if renorm else a)) for a in s])
        num = (L[:E] - L[E:]) / (2 * h)
        lg, _ = _logits(x[None], False)
        d = torch.empty(1, E, device="cuda")
        G.moe_router_topk_bwd(lg, 1, E, k, r, torch.from_numpy(ids0).cuda(), torch.from_numpy(dw[None]).cuda(), d)
        torch.cuda.synchronize()
        assert np.max(np.abs(d.cpu().numpy()[0] - num)) <= h * h / 6 * 10 * np.abs(dw).sum() + 1e-5


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_small_scores_beside_a_bias(G, score):
    """A bias that decides for experts whose scores fp32 does not hold, or only just: their weights are still the
    ratios of the scores."""
    E = 64
    rng = np.random.default_rng(14)
    x = (rng.standard_normal((24, E)) * 2).astype(np.float32)
    x[:, :8] -= np.linspace(0, 230, 24, dtype=np.float32)[:, None]
    bias = np.where(np.arange(E) < 8, 2.0, 0.0).astype(np.float32)
    _run(G, x, 4, False, bias, None, score=score)
    _run(G, x, 4, False, bias, None, score=score, renorm=False)
