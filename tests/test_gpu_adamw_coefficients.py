"""The step's coefficients, whose errors are the same for every element and add up
over the steps: weight decay far below an fp32 rounding of 1.

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
