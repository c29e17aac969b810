"""The AdamW step, its 8-bit states and the gradients' norm on the GPU against the
float64 oracle.

Tolerances, U = 2^-24.  fp32 states: the coefficient, the product and the sum are
each off by U, so 4 U (|b1 m| + |(1 - b1) g|) for m and, with the square and the
scaled gradient, 7 U of v' for v.  The parameter: p (1 - a decay) is off by 3 U
|p|; the update a m' / (...) by what m' is off by over its denominator, half of
what v' is off by, and 10 roundings, 20 U in all beside m's; the difference by U.
bf16 parameters add half a step, 2^-8 of the value.  8-bit scales are
the roundings of the blocks' largest values, to half a step and 2^-48 of the
value: with beta1 = 0.9 a value (9 m + g) / 10 of fp32 m and bf16 g lies on the
middle between two fp32 values one time in ten, and the roundings in 64 bits
before it, 4 of 2^-53 each at most, decide for either.  Codes are equal, given the
scales.  The norm is a sum in 64 bits: one rounding to fp32, 1.01 U; the factor
has one more."""
import numpy as np
import pytest

import workloads as W
from oracle import formats as F
from oracle import training as P
from tests.test_gpu_lora import G  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=7)


def to_dev(a):
    import torch
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).cuda().view(torch.bfloat16)
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def to_host(t):
    import torch
    if t.dtype == torch.bfloat16:
        return F.bf16_bits_to_f64(t.view(torch.int16).cpu().numpy().view(np.uint16))
    return t.cpu().numpy()


class Tensor:
    """One tensor of a step: host copies, device copies with a guard behind, the plan's struct."""

    def __init__(self, G, seed, n, param="fp32", bf16_grad=False, bits=32, weight_decay=0.01, lr_scale=1.0, fresh=False):  # noqa: F811
        import torch
        rng = np.random.default_rng(seed)
        self.n, self.bits, self.kind, self.decay, self.lr_scale = n, bits, param, weight_decay, lr_scale
        f32 = lambda std: (rng.standard_normal(n) * std).astype(np.float32)  # noqa: E731
        spread = np.exp(rng.standard_normal((n + 127) // 128))[np.arange(n) // 128]
        p, g = f32(0.05), (f32(1e-2) * spread).astype(np.float32)
        self.h = {"grad": W.to_bf16_bits(g) if bf16_grad else g}
        self.h["param"] = p if param == "fp32" else W.to_bf16_bits(p)
        if param == "master":
            self.h["master"] = p
        m, v = (f32(3e-3) * spread).astype(np.float32), ((f32(1e-2) * spread) ** 2).astype(np.float32)
        if fresh:
            m[:], v[:] = 0, 0
        if bits == 32:
            self.h |= {"m": m, "v": v}
        else:
            cm, ms, cv, vs = P.state8_encode(m.astype(np.float64), v.astype(np.float64))
            self.h |= {"m": cm, "v": cv, "m_scale": ms, "v_scale": vs}
        self.d, self.guard = {}, {}
        for k, a in self.h.items():
            t = to_dev(np.concatenate([a, np.full(64, 77, a.dtype)]))
            self.d[k], self.guard[k] = t[:len(a)], t[len(a):]
        self.struct = G.adamw_tensor(self.d["param"], self.d["grad"], self.d["m"], self.d["v"],
                                     master=self.d.get("master"), m_scale=self.d.get("m_scale"),
                                     v_scale=self.d.get("v_scale"), weight_decay=weight_decay, lr_scale=lr_scale)

    def f64(self, k):
        a = self.h[k]
        return F.bf16_bits_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)

    def check(self, hyper, grad_scale=1.0):
        hy = {**HYPER, **hyper}
        lr = hy["lr"] * float(np.float32(self.lr_scale))
        b1, b2, t = hy["beta1"], hy["beta2"], hy["step"]
        decay = float(np.float32(self.decay))
        if self.bits == 8:
            m0, v0 = P.state8_decode(self.h["m"], self.h["m_scale"], self.h["v"], self.h["v_scale"])
        else:
            m0, v0 = self.f64("m"), self.f64("v")
        old = self.f64("master" if self.kind == "master" else "param")
        g = self.f64("grad") * float(grad_scale)
        p, m, v = P.adamw(old, self.f64("grad"), m0, v0, lr, b1, b2, hy["eps"], t, decay, grad_scale)
        got = {k: to_host(a) for k, a in self.d.items()}
        for k, a in self.guard.items():
            want = np.full(64, 77, self.h[k].dtype)
            assert np.array_equal(to_host(a), F.bf16_bits_to_f64(want) if want.dtype == np.uint16 else want), k
        tol_m = 4 * U * (np.abs(b1 * m0) + np.abs((1 - b1) * g)) + 1e-44
        if self.bits == 32:
            assert np.all(np.abs(got["m"] - m) <= tol_m)
            assert np.all(np.abs(got["v"] - v) <= 7 * U * v + 1e-44)
        else:
            for k, value in (("m_scale", np.abs(m)), ("v_scale", np.sqrt(v))):
                top = np.maximum.reduceat(value, np.arange(0, self.n, 128))
                assert np.all(np.abs(got[k] - top) <= np.spacing(top.astype(np.float32)) / 2.0 + 2.0 ** -48 * top), k
            cm, _, cv, _ = P.state8_encode(m, v, (got["m_scale"], got["v_scale"]))
            assert np.array_equal(got["m"], cm) and np.array_equal(got["v"], cv)
        denom = np.sqrt(v / (1 - b2 ** t)) + hy["eps"]
        coef = abs(lr) / (1 - b1 ** t)
        update = np.abs(old * (1 - lr * decay) - p)
        tol = 4 * U * np.abs(old) + coef * tol_m / denom + 20 * U * update + U * np.abs(p) + 1e-44
        if self.kind == "master":
            assert np.all(np.abs(got["master"] - p) <= tol)
        bf16 = 0 if self.kind == "fp32" else 2.0 ** -8 * 1.01
        assert np.all(np.abs(got["param"] - p) <= tol + bf16 * np.abs(p)), self.kind
        if self.kind == "master":                          # the rounding of the master
            assert np.array_equal(got["param"], F.bf16_bits_to_f64(W.to_bf16_bits(got["master"])))


KINDS = [(p, g, b) for p in ("fp32", "bf16", "master") for g in (False, True) for b in (32, 8)]


@pytest.mark.parametrize("param,bf16_grad,bits", KINDS)
def test_sizes(G, param, bf16_grad, bits):  # noqa: F811
    import torch
    sizes = [1, 2, 3, 4, 5, 127, 128, 129, 255, 1000, 1023, 1024, 1025, 4095, 4096, 4097, 12289, 20000]
    ts = [Tensor(G, i, n, param, bf16_grad, bits, weight_decay=0.01 * (i % 3), lr_scale=0.5 + i % 2)
          for i, n in enumerate(sizes)]
    G.moe_adamw_step(G.adamw_plan([t.struct for t in ts]), G.adamw(**HYPER))
    torch.cuda.synchronize()
    for t in ts:
        t.check({})


def test_every_kind_in_one_plan(G):  # noqa: F811
    import torch
    ts = [Tensor(G, i, 300 * i + 5, p, g, b) for i, (p, g, b) in enumerate(KINDS)]
    empty = torch.empty(0, device="cuda")
    none = [G.adamw_tensor(None, torch.ones(70, device="cuda"), None, None), G.adamw_tensor(empty, empty, empty, empty)]
    scale = torch.tensor([0.25], device="cuda")
    G.moe_adamw_step(G.adamw_plan([none[0]] + [t.struct for t in ts] + none[1:]), G.adamw(**HYPER, grad_scale=scale))
    torch.cuda.synchronize()
    for t in ts:
        t.check({}, grad_scale=0.25)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("hyper", [dict(beta1=0.0), dict(beta2=0.0), dict(step=1), dict(step=100000), dict(eps=1e-3),
                                   dict(lr=0.0), dict(lr=-1e-3)])
def test_numbers(G, bits, hyper):  # noqa: F811
    import torch
    t = Tensor(G, 3, 1500, "master", bits=bits, fresh=hyper.get("step") == 1)
    G.moe_adamw_step(G.adamw_plan([t.struct]), G.adamw(**{**HYPER, **hyper}))
    torch.cuda.synchronize()
    t.check(hyper)


@pytest.mark.parametrize("bits", [32, 8])
def test_numbers_of_the_device(G, bits):  # noqa: F811
    """Step and learning rate read on the device; a step below 1 counts as 1."""
    import torch
    for step, used in ((12, 12), (0, 1), (-5, 1)):
        t = Tensor(G, 4, 3000, "fp32", bits=bits)
        lr = torch.tensor([0.03125], device="cuda")
        G.moe_adamw_step(G.adamw_plan([t.struct]), G.adamw(7.0, 0.9, 0.99, 1e-8, step=0, lr_dev=lr,
                                                          step_dev=torch.tensor([step], dtype=torch.int32, device="cuda")))
        torch.cuda.synchronize()
        t.check(dict(lr=0.03125, step=used))


@pytest.mark.parametrize("bits", [32, 8])
def test_no_step_without_a_norm(G, bits):  # noqa: F811
    import torch
    t = Tensor(G, 5, 2000, "master", bits=bits)
    G.moe_adamw_step(G.adamw_plan([t.struct]), G.adamw(**HYPER, grad_scale=torch.tensor([float("nan")], device="cuda")))
    torch.cuda.synchronize()
    for k, a in t.d.items():
        assert np.array_equal(to_host(a), t.f64(k) if t.h[k].dtype == np.uint16 else t.h[k]), k


def test_many_steps_of_8_bits(G):  # noqa: F811
    """Each step's codes follow from the codes before it, to the bit; a block that only decays keeps its codes while
    its scales fall; a block of zeros stays zero; elements far below the block's largest keep a second moment."""
    import torch
    t = Tensor(G, 6, 128 * 6 + 9, "master", bits=8)
    t.d["grad"][:128] = 0
    t.d["grad"][128:256] = 0
    t.d["m"][128:256] = 0
    t.d["v"][128:256] = 0
    t.d["m_scale"][1] = 0
    t.d["v_scale"][1] = 0
    t.d["grad"][256:384] *= torch.logspace(0, -12, 128, device="cuda")
    plan = G.adamw_plan([t.struct])
    for step in range(1, 6):
        for k in t.h:
            a = t.d[k]
            t.h[k] = (a.view(torch.int16).cpu().numpy().view(np.uint16) if a.dtype == torch.bfloat16 else a.cpu().numpy()).copy()
        G.moe_adamw_step(plan, G.adamw(**{**HYPER, "step": step}))
        torch.cuda.synchronize()
        t.check(dict(step=step))
        assert np.array_equal(t.h["m"][:128], to_host(t.d["m"][:128])) and np.array_equal(t.h["v"][:128], to_host(t.d["v"][:128]))
        assert float(t.d["m_scale"][0]) < t.h["m_scale"][0] and float(t.d["v_scale"][0]) < t.h["v_scale"][0]
        assert torch.all(t.d["m"][128:256] == 0) and torch.all(t.d["v"][128:256] == 0)
        assert torch.all((t.d["v"][256:384] > 0) | (t.d["grad"][256:384] == 0))


def test_values_that_are_not_finite(G):  # noqa: F811
    """8 bits: the block's scales become NaN, its codes 0; the other blocks and tensors go on."""
    import torch
    for value in (float("nan"), float("inf"), -float("inf")):
        t, other = Tensor(G, 7, 700, "master", bits=8), Tensor(G, 8, 700, "fp32", bits=32)
        t.d["grad"][200] = value
        G.moe_adamw_step(G.adamw_plan([t.struct, other.struct]), G.adamw(**HYPER))
        torch.cuda.synchronize()
        t.h["grad"][200] = value
        other.check({})
        ms, vs = to_host(t.d["m_scale"]), to_host(t.d["v_scale"])
        assert np.array_equal(np.isnan(ms), np.arange(6) == 1) and np.array_equal(np.isnan(vs), np.arange(6) == 1)
        assert torch.all(t.d["m"][128:256] == 0) and torch.all(t.d["v"][128:256] == 0)
        p = to_host(t.d["master"])
        assert not np.isfinite(p[200]) and np.all(np.isfinite(np.delete(p, 200)))


def test_large_and_small_values(G):  # noqa: F811
    import torch
    for std in (1e-30, 1e-18, 1e18):
        t = Tensor(G, 9, 1000, "fp32", bits=8, fresh=True)
        t.h["grad"] = (t.h["grad"] / np.float32(1e-2) * np.float32(std)).astype(np.float32)
        t.d["grad"].copy_(torch.from_numpy(t.h["grad"]))
        G.moe_adamw_step(G.adamw_plan([t.struct]), G.adamw(**HYPER))
        torch.cuda.synchronize()
        m, v = 0.1 * t.f64("grad"), 0.01 * t.f64("grad") ** 2
        cm, ms, cv, vs = P.state8_encode(m, v)
        assert np.array_equal(to_host(t.d["m"]), cm) and np.array_equal(to_host(t.d["v"]), cv)
        assert np.array_equal(to_host(t.d["m_scale"]), ms) and np.array_equal(to_host(t.d["v_scale"]), vs)


@pytest.mark.parametrize("eps", [0.0, 1e-18, 1e-15, 1e-12])
def test_small_roots(G, eps):  # noqa: F811
    """Second moments below fp32's normal numbers, beside an eps that they still change (v' keeps 10 bits there, its
    root 2^-11 of an eighth of eps or less; with eps 0 they are normal)."""
    import torch
    std = 1e-19 if eps else 1e-16
    t = Tensor(G, 10, 1000, "fp32", fresh=True)
    t.h["param"][:] = 0
    t.h["grad"] = (np.sign(t.h["grad"]) * (std + np.abs(t.h["grad"]) * std)).astype(np.float32)
    t.d["param"].zero_()
    t.d["grad"].copy_(torch.from_numpy(t.h["grad"]))
    G.moe_adamw_step(G.adamw_plan([t.struct]), G.adamw(**{**HYPER, "eps": eps}))
    torch.cuda.synchronize()
    v = 0.01 * t.f64("grad") ** 2 / (1 - 0.99 ** 7)
    if 0 < eps <= 1e-18:                       # what v' loses below 2^-126: half of 2^-149
        got, m = to_host(t.d["param"]), 0.1 * t.f64("grad") / (1 - 0.9 ** 7)
        want = -2e-3 * m / (np.sqrt(v) + eps)
        assert np.all(np.abs(got - want) <= (24 * U + 2.0 ** -150 / (0.01 * t.f64("grad") ** 2)) * np.abs(want))
    else:
        t.check({"eps": eps})


@pytest.mark.parametrize("n", [0, 1, 5, 127, 128, 130, 1000, 5000])
def test_unpack(G, n):  # noqa: F811
    import torch
    rng = np.random.default_rng(n)
    cm, cv = rng.integers(-127, 128, n).astype(np.int8), rng.integers(0, 256, n).astype(np.uint8)
    blocks = (n + 127) // 128
    ms, vs = rng.random(blocks).astype(np.float32), (rng.random(blocks) * 1e-3).astype(np.float32)
    m, v = torch.full((n + 3,), -7.0, device="cuda"), torch.full((n + 3,), -7.0, device="cuda")
    G.moe_adamw_unpack(to_dev(cm), to_dev(ms), to_dev(cv), to_dev(vs), n, m, v)
    torch.cuda.synchronize()
    wm, wv = P.state8_decode(cm, ms, cv, vs)
    assert np.all(np.abs(to_host(m)[:n] - wm) <= 1.01 * U * np.abs(wm)) and np.all(to_host(m)[n:] == -7)
    assert np.all(np.abs(to_host(v)[:n] - wv) <= 1.01 * U * np.abs(wv) + 1e-45) and np.all(to_host(v)[n:] == -7)
    m2 = torch.empty(max(1, n), device="cuda")
    G.moe_adamw_unpack(to_dev(cm), to_dev(ms), None, None, n, m_out=m2)
    torch.cuda.synchronize()
    assert torch.equal(m2[:n], m[:n])


def _norm(G, tensors, max_norm=1.0, plan=None):  # noqa: F811
    import torch
    out = torch.full((3,), -7.0, device="cuda")
    ws = torch.full((G.moe_grad_norm_workspace_bytes(),), 0xFF, dtype=torch.uint8, device="cuda")
    G.moe_grad_norm(plan or G.adamw_plan([G.adamw_tensor(None, t, None, None) for t in tensors]), max_norm, out, ws)
    torch.cuda.synchronize()
    got = out.cpu().numpy()
    assert got[2] == -7
    return got[:2]


@pytest.mark.parametrize("sizes", [[], [0], [1], [3, 0, 4], [5, 128, 4097, 1], [9] * 1500, [5000000, 77]])
@pytest.mark.parametrize("bf16", [False, True])
def test_norm(G, sizes, bf16):  # noqa: F811
    rng = np.random.default_rng(len(sizes))
    host = [(rng.standard_normal(n) * 0.1).astype(np.float32) for n in sizes]
    host = [W.to_bf16_bits(a) if bf16 else a for a in host]
    f64 = [F.bf16_bits_to_f64(a) if bf16 else a.astype(np.float64) for a in host]
    for max_norm in (0.5, 1e6, float("inf")):
        got = _norm(G, [to_dev(a) for a in host], max_norm)
        norm, factor = P.grad_norm([a if len(a) < 100000 else [np.sqrt(np.sum(a * a))] for a in f64], max_norm)
        assert abs(got[0] - norm) <= 1.01 * U * norm and abs(got[1] - factor) <= 2.01 * U * factor


@pytest.mark.parametrize("sizes", [[40000, 3, 20000], [2048] * 31, [65536], [65537], [1] * 32, [1] * 33])
def test_norm_of_few_pieces(G, sizes):  # noqa: F811
    """One workgroup's plans and the ones after them, to their extremes."""
    import torch
    test_norm(G, sizes, False)
    test_norm(G, sizes, True)
    for bad in (float("nan"), float("inf"), 3e38):
        t = [torch.ones(n, device="cuda") for n in sizes]
        t[-1][-1] = bad
        t[0][0] = 3e38 if bad == 3e38 else 1
        got = _norm(G, t)
        assert not np.isfinite(got[0]) and np.isnan(got[1])


def test_norm_extremes(G):  # noqa: F811
    import torch
    got = _norm(G, [torch.full((1000,), 1e30, device="cuda")])
    assert abs(got[0] / (np.float64(np.float32(1e30)) * np.sqrt(1000)) - 1) <= 1.01 * U
    got = _norm(G, [torch.full((7,), 1e-40, device="cuda")])
    assert got[0] > 0 and got[1] == 1
    for bad in (float("nan"), float("inf"), 3e38):           # the last: a norm beyond fp32
        got = _norm(G, [torch.full((5,), bad, device="cuda"), torch.ones(9, device="cuda")])
        assert not np.isfinite(got[0]) and np.isnan(got[1])


def test_plan_follows_contents(G):  # noqa: F811
    """A plan holds addresses: contents may change between calls."""
    import torch
    g = torch.ones(5000, device="cuda")
    plan = G.adamw_plan([G.adamw_tensor(None, g, None, None)])
    assert abs(_norm(G, None, plan=plan)[0] - np.sqrt(5000)) < 1e-4
    g.fill_(2.0)
    assert abs(_norm(G, None, plan=plan)[0] - 2 * np.sqrt(5000)) < 1e-4


def test_clip_and_step(G):  # noqa: F811
    """The factor goes from one call to the next on the device."""
    import torch
    t = Tensor(G, 10, 6000, "master", bits=8)
    plan = G.adamw_plan([t.struct])
    out, ws = torch.empty(2, device="cuda"), torch.empty(G.moe_grad_norm_workspace_bytes(), dtype=torch.uint8, device="cuda")
    G.moe_grad_norm(plan, 0.1, out, ws)
    G.moe_adamw_step(plan, G.adamw(**HYPER, grad_scale=out[1:]))
    torch.cuda.synchronize()
    norm, factor = P.grad_norm([t.h["grad"]], 0.1)
    got = float(out[1])
    assert abs(got - factor) <= 2.01 * U * factor and factor < 1
    t.check({}, grad_scale=got)
