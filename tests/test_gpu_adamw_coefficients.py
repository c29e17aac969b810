"""The step's coefficients, whose errors are the same for every element and add up
over the steps: weight decay far below an fp32 rounding of 1, and betas near 1.

A single fp32 result is off by up to half a step, which hides them; the mean over n
elements is not.  The results lie in [1, 2) (some at its ends' other sides, with
half or twice the step), 2^-23 apart, and fall anywhere between two of them: a
rounding has a deviation of 2^-23 / sqrt(12), the mean of n = 2^20 of them 1/1024 of
that, 3.4e-11.  Six deviations are 2.1e-10; values of [2, 4) among them, fewer than
1% here, and the roundings of the small terms, whose signs vary, stay within 2.5e-10."""
import numpy as np
import pytest

import workloads as W
from oracle import training as P
from tests.test_gpu_adamw import to_dev, to_host
from tests.test_gpu_lora import G  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
N = 1 << 20
MEAN = 2.5e-10


def one_to_two(rng):
    return (1 + rng.integers(0, 1 << 23, N) * 2.0 ** -23).astype(np.float32)


@pytest.mark.parametrize("kind,bits", [("fp32", 32), ("master", 32), ("fp32", 8), ("master", 8)])
@pytest.mark.parametrize("decay", [1e-2, 1e-3, -1e-3])
def test_small_decay(G, kind, bits, decay):  # noqa: F811
    """lr decay of 1e-7 and 1e-8: p (1 - 1e-8) would be p, and p (1 - 1e-7) p (1 - 1.19e-7)."""
    import torch
    rng = np.random.default_rng(1)
    p = one_to_two(rng)
    d = {"param": to_dev(p) if kind == "fp32" else to_dev(W.to_bf16_bits(p))}
    master = to_dev(p) if kind == "master" else None
    # updates of a few steps of p, of either sign
    if bits == 32:
        m, v = (rng.standard_normal(N) * 0.05).astype(np.float32), np.ones(N, np.float32)
        scales = {}
        m0, v0 = m.astype(np.float64), v.astype(np.float64)
    else:
        m, v = rng.integers(-127, 128, N).astype(np.int8), np.full(N, 255, np.uint8)
        ms, vs = np.full(N // 128, 0.2, np.float32), np.ones(N // 128, np.float32)
        m0, v0 = P.state8_decode(m, ms, v, vs)
        scales = dict(m_scale=to_dev(ms), v_scale=to_dev(vs))
    grad = torch.zeros(N, device="cuda")
    plan = G.adamw_plan([G.adamw_tensor(d["param"], grad, to_dev(m), to_dev(v), master=master, weight_decay=decay, **scales)])
    hyper = dict(lr=1e-5, beta1=0.9, beta2=0.99, eps=1e-8, step=5000)
    G.moe_adamw_step(plan, G.adamw(**hyper))
    torch.cuda.synchronize()
    want, _, _ = P.adamw(p, np.zeros(N), m0, v0, 1e-5, 0.9, 0.99, 1e-8, 5000, float(np.float32(decay)))
    got = to_host(d["param"] if master is None else master).astype(np.float64)
    assert abs(np.mean(got - want.astype(np.float32))) <= MEAN
    assert np.all(np.abs(got - want) <= 2.0 ** -23 * 1.01)


@pytest.mark.parametrize("beta1,beta2", [(0.9, 0.999), (0.95, 0.99999), (1 - 1e-5, 1 - 2e-8), (1 - 1e-6, 1 - 2.0 ** -30)])
def test_betas_near_one(G, beta1, beta2):  # noqa: F811
    """The moments of 32 bits: beta and 1 - beta add up to 1, also where fp32's beta is 1 itself."""
    import torch
    rng = np.random.default_rng(2)
    m, v = one_to_two(rng), one_to_two(rng)
    # gradients of either sign whose squares add between 0 and 64 steps to v, each as likely
    g = np.sqrt(rng.random(N) * 2.0 ** -17 / (1 - beta2)) * rng.choice([-1.0, 1.0], N)
    g = g.astype(np.float32)
    dm, dv = to_dev(m), to_dev(v)
    param = torch.zeros(N, device="cuda")
    G.moe_adamw_step(G.adamw_plan([G.adamw_tensor(param, to_dev(g), dm, dv)]), G.adamw(1e-3, beta1, beta2, 1e-8, step=100))
    torch.cuda.synchronize()
    _, want_m, want_v = P.adamw(np.zeros(N), g, m, v, 1e-3, beta1, beta2, 1e-8, 100)
    for got, want, old, add in ((to_host(dm), want_m, m, (1 - beta1) * g.astype(np.float64)),
                                (to_host(dv), want_v, v, (1 - beta2) * g.astype(np.float64) ** 2)):
        err = got.astype(np.float64) - want
        # (1 - beta's own rounding, 2^-24 of the term, is the same for all too)
        assert abs(np.mean(err)) <= MEAN + 2.0 ** -24 * abs(np.mean(add)), (np.mean(err), np.mean(add))
        assert np.all(np.abs(err) <= 2.0 ** -23 * (np.abs(old) + 4 * np.abs(add)))


@pytest.mark.parametrize("beta1,beta2", [(0.9, 0.999), (0.95, 0.99999), (0.0, 0.0), (0.99, 0.98)])
def test_infinite_moments_stay(G, beta1, beta2):  # noqa: F811
    """Moments that left fp32 (a gradient past 1.8e19 leaves an infinite v beside a finite m) stay infinite, whichever
    way beta rounds, and the parameter of such a v stays put."""
    import torch
    inf = float("inf")
    m, v = torch.tensor([inf, -inf, 1.0, 0.0], device="cuda"), torch.tensor([1.0, 1.0, inf, inf], device="cuda")
    param = torch.ones(4, device="cuda")
    plan = G.adamw_plan([G.adamw_tensor(param, torch.ones(4, device="cuda"), m, v)])
    for step in (1, 2, 3):
        G.moe_adamw_step(plan, G.adamw(1e-3, beta1, beta2, 1e-8, step=step))
        torch.cuda.synchronize()
        if beta1:
            assert m[0] == inf and m[1] == -inf and param[0] == -inf and param[1] == inf
        if beta2:
            assert v[2] == inf and v[3] == inf and param[2] == 1 and param[3] == 1


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("decay", [0.0, 0.1, -0.1])
def test_infinite_parameters_stay(G, decay, bits):  # noqa: F811
    """A parameter that left fp32 stays infinite, with or without a decay, and a NaN a NaN."""
    import torch
    inf = float("inf")
    start = torch.tensor([inf, -inf, float("nan"), 3.4e38, -3.4e38], device="cuda")
    for grad in (1.0, 0.0, -1.0):
        param, g = start.clone(), torch.full((5,), grad, device="cuda")
        if bits == 32:
            t = G.adamw_tensor(param, g, torch.zeros(5, device="cuda"), torch.zeros(5, device="cuda"), weight_decay=decay)
        else:
            t = G.adamw_tensor(param, g, torch.zeros(5, dtype=torch.int8, device="cuda"), torch.zeros(5, dtype=torch.uint8, device="cuda"),
                               m_scale=torch.zeros(1, device="cuda"), v_scale=torch.zeros(1, device="cuda"), weight_decay=decay)
        G.moe_adamw_step(G.adamw_plan([t]), G.adamw(1e-3))
        torch.cuda.synchronize()
        assert param[0] == inf and param[1] == -inf and torch.isnan(param[2])
        assert abs(float(param[3]) / 3.4e38 - (1 - 1e-3 * decay)) <= 1e-6 and param[4] == -param[3]
