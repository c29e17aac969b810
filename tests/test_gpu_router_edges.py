"""The router and its gradient where 32 bits do not hold what decides: NaN and
infinities in the bias, groups whose two best values cancel, scores and
scales near the end of fp32, chosen experts far below the row's largest logit.
Against the float64 oracle, with the tolerances of test_gpu_router."""
import numpy as np
import pytest

from oracle import operators as P
from tests.test_gpu_router import G, U, _logits, _run  # noqa: F401  (G: the fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- NaN and infinities in the bias
# (a quad with a NaN: its one number must not count twice; the group sizes of the kernels in 32 bits and, E % 4
# != 0 or groups of 3, in 64; up to and past 2048 tokens)
@pytest.mark.parametrize("T", [40, 2100])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_score", ["top2", "max"])
@pytest.mark.parametrize("E,k,groups,keep", [(16, 3, 4, 1), (64, 4, 4, 2), (12, 3, 4, 2), (256, 8, 8, 3)])
def test_router_nan_bias(G, E, k, groups, keep, group_score, score, bf16, T):  # noqa: F811
    rng = np.random.default_rng(E + groups)
    size = E // groups
    x = rng.standard_normal((T, E)).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.3).astype(np.float32)
    x[:, 0] += 3.0                                  # the number beside the NaN is its group's best
    bias[1] = np.nan
    bias[2 * size:3 * size] = np.nan                # a group of NaN alone
    bias[3 * size + size // 2:4 * size] = np.nan    # half a group
    _run(G, x, k, bf16, bias, None, score=score, n_groups=groups, topk_groups=keep, group_score=group_score)


def test_router_nan_bias_worked_case(G):  # noqa: F811
    """Group 0: 0.88 beside 0.5; group 1: twice 0.73.  The second is chosen."""
    x = np.zeros((1, 16), np.float32)
    x[0, 0], x[0, 3], x[0, 4], x[0, 5] = 2.0, -0.5, 1.0, 1.0
    x[0, 8:] = -5.0
    bias = np.zeros(16, np.float32)
    bias[1] = np.nan
    _run(G, x, 2, False, bias, None, score="sigmoid", n_groups=4, topk_groups=1, group_score="top2")


@pytest.mark.parametrize("group_score", ["top2", "max"])
@pytest.mark.parametrize("groups,keep", [(1, 1), (4, 2), (4, 3)])
@pytest.mark.parametrize("T", [30, 2100])
def test_router_infinite_and_nan_bias(G, T, groups, keep, group_score):  # noqa: F811
    E = 32
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, E)).astype(np.float32)
    for put in ({3: -np.inf}, {3: np.inf, 9: np.inf}, {3: np.inf, 4: -np.inf, 8: np.nan}, {e: -np.inf for e in range(8, 24)},
                {e: -np.inf for e in range(E)}, {e: np.nan for e in range(E)}):
        bias = np.zeros(E, np.float32)
        for e, v in put.items():
            bias[e] = v
        _run(G, x, 5, False, bias, None, score="sigmoid", n_groups=groups, topk_groups=keep, group_score=group_score)


# ---------------------------------------------------------------- groups whose two best values cancel
@pytest.mark.parametrize("T", [2000, 4096])
@pytest.mark.parametrize("big", [1000.0, 30000.0])
def test_router_groups_of_large_opposite_choice_values(G, T, big):  # noqa: F811
    """Group 0's two best choice values are about +big and -big, so that in 32
    bits each is off by up to big 2^-24 and so is their sum, of about 1; group
    1's are scores alone.  The sums differ by up to twice that."""
    rng = np.random.default_rng(int(big) + T)
    x = rng.uniform(-1.0, 0.0, (T, 8))
    s = 1 / (1 + np.exp(-x))
    need = s[:, 0] + s[:, 1] + rng.uniform(-1, 1, T) * big * 2.0 ** -23 - s[:, 4]     # the score of expert 5
    x[:, 5] = np.log(need / (1 - need))
    x[:, [2, 3, 6, 7]] = -9.0
    bias = np.array([big, -big, -4 * big, -4 * big, 0, 0, 0, 0], np.float32)
    _run(G, x.astype(np.float32), 2, False, bias, None, score="sigmoid", n_groups=2, topk_groups=1, group_score="top2")


# ---------------------------------------------------------------- scores and scales that fp32 does not hold
@pytest.mark.parametrize("renorm", [True, False])
def test_router_gradient_of_small_sigmoid_scores(G, renorm):  # noqa: F811
    """Every chosen score below, at and above what fp32 holds: the forward's weights are ratios of scores in 64
    bits, and so is the gradient."""
    rng = np.random.default_rng(1)
    E, k = 24, 4
    top = np.array([-5, -30, -60, -70, -80, -87, -87.5, -88.0, -88.4, -88.8, -90, -100, -104, -120, -200, -500, -700],
                   np.float32)
    x = top[:, None] - rng.uniform(0, 3, (len(top), E)).astype(np.float32)
    _run(G, x, k, False, None, rng.standard_normal((len(top), k)), score="sigmoid", renorm=renorm, scale=2.5)
    # some chosen scores small, others not
    x[:, :2] = rng.standard_normal((len(top), 2))
    _run(G, x, k, False, None, rng.standard_normal((len(top), k)), score="sigmoid", renorm=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_gradient_of_small_scores_beside_a_bias(G, score):  # noqa: F811
    E = 64
    rng = np.random.default_rng(14)
    x = (rng.standard_normal((24, E)) * 2).astype(np.float32)
    x[:, :8] -= np.linspace(0, 230, 24, dtype=np.float32)[:, None]
    bias = np.where(np.arange(E) < 8, 2.0, 0.0).astype(np.float32)
    for renorm in (True, False):
        _run(G, x, 4, False, bias, rng.standard_normal((24, 4)), score=score, renorm=renorm)


def test_router_gradient_of_large_weight_gradients(G):  # noqa: F811
    """dweights / S passes fp32's range, the gradient does not."""
    rng = np.random.default_rng(3)
    x = -60 - rng.uniform(0, 2, (6, 8)).astype(np.float32)
    _run(G, x, 3, False, None, rng.standard_normal((6, 3)) * 1e15, score="sigmoid", scale=2.0)


@pytest.mark.parametrize("group_score", [None, "top2"])
def test_router_gradient_is_zero_where_the_weights_are(G, group_score):  # noqa: F811
    """Chosen for their bias alone, with logits so far below the row's largest that their scores are 0 in 64 bits
    (as under a mask of the type's lowest value): weights and gradient are 0."""
    import torch
    rng = np.random.default_rng(4)
    E, k, T = 16, 3, 8
    x = rng.standard_normal((T, E)).astype(np.float32)
    x[:, :8] = np.array([np.finfo(np.float32).min, -1e4, -800, -760], np.float32).repeat(2)[:, None]
    x[:, :8] -= np.arange(8, dtype=np.float32)
    bias = np.where(np.arange(E) < 8, 4.0, 0.0).astype(np.float32)
    kw = dict(score="softmax", renorm=True)
    if group_score:
        kw.update(n_groups=4, topk_groups=2, group_score=group_score)
    _, w = P.router_topk(x.astype(np.float64), k, bias=bias, **kw)
    assert np.all(w == 0)
    _run(G, x, k, False, bias, rng.standard_normal((T, k)), **kw)
    # and just above: ratios again
    x[:, :8] = -300.0 - rng.uniform(0, 3, (T, 8))
    _run(G, x, k, False, bias, rng.standard_normal((T, k)), **kw)
    # the ids alone decide, whoever chose them: the same rows without groups and bias in the struct keep the rule of
    # a softmax over the chosen logits
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda") + torch.arange(k, dtype=torch.int32, device="cuda")
    lg, v = _logits(x, False)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    d = torch.full((T, E), 7.0, device="cuda")
    G.moe_router_topk_bwd(lg, T, E, k, G.router(**dict(score="softmax", renorm=True)), ids, torch.from_numpy(dw).cuda(), d)
    torch.cuda.synchronize()
    want = P.router_topk_bwd(v, ids.cpu().numpy(), dw.astype(np.float64))
    assert np.max(np.abs(d.double().cpu().numpy() - want)) <= 4 * (2 * 3 + 32) * U * 2 * np.abs(dw).sum(1).max()


@pytest.mark.parametrize("scale", [1e-20, -1e-28, 1e30, 0.0])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_router_scale_and_small_scores(G, score, scale):  # noqa: F811
    """scale * score passes fp32's range, scale * weight does not."""
    rng = np.random.default_rng(5)
    E = 32
    x = (rng.standard_normal((20, E)) * 2).astype(np.float32)
    x[:, :8] -= np.linspace(0, 66, 20, dtype=np.float32)[:, None]
    bias = np.where(np.arange(E) < 8, 2.0, 0.0).astype(np.float32)
    _run(G, x, 4, False, bias, None, score=score, scale=scale)
    x[:, 8:] -= np.linspace(0, 66, 20, dtype=np.float32)[:, None]
    _run(G, x, 4, False, None, None, score=score, scale=scale)


# ---------------------------------------------------------------- every width of the groups' merges
@pytest.mark.parametrize("T", [30, 2100])
@pytest.mark.parametrize("E,groups,keep", [(256, 64, 20), (256, 32, 9), (256, 16, 5), (256, 8, 3), (256, 4, 2), (256, 2, 1),
                                           (512, 2, 1), (512, 8, 7), (1024, 4, 3), (1024, 8, 2), (96, 3, 2), (640, 5, 2)])
def test_router_group_widths(G, T, E, groups, keep):  # noqa: F811
    """Groups of 4 to 256 experts, in 16, 32 and 64 lanes per token."""
    rng = np.random.default_rng(E + groups)
    x = rng.standard_normal((T, E))
    bias = (rng.standard_normal(E) * 0.3).astype(np.float32)
    _run(G, x, 6, False, bias, None, score="sigmoid", n_groups=groups, topk_groups=keep, group_score="top2")
    _run(G, x, 6, True, None, None, score="softmax", n_groups=groups, topk_groups=keep, group_score="max")
