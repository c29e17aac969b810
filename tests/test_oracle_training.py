"""Pins of the oracle of adapters, AdamW and the norm: loops, closed forms,
finite differences, exhaustive searches.  CPU only."""
import math

import numpy as np
import pytest

import workloads as W
from oracle import formats as F
from oracle import training as P


def _bits(rng, *shape):
    return W.to_bf16_bits(rng.standard_normal(shape).astype(np.float32))


def _case(src=True):
    rng = np.random.default_rng(0)
    T, r, K, N, counts = 7, 8, 16, 24, [3, 0, 2]
    t = dict(x=_bits(rng, T, K), A=_bits(rng, 3, r, K), B=_bits(rng, 3, N, r), base=_bits(rng, T, N),
             scale=rng.random(3).astype(np.float32))
    return t, counts, (np.array([6, 0, 3, 9, 5], dtype=np.int32) if src else None), rng


@pytest.mark.parametrize("with_src", [True, False])
def test_lora_against_loops(with_src):
    t, counts, src, _ = _case(with_src)
    u, y = P.lora_fwd(t["x"], t["A"], t["B"], t["scale"], counts, 5, src, t["base"])
    f = {k: F.bf16_bits_to_f64(v) for k, v in t.items() if k != "scale"}
    written = set()
    for g in range(5):
        e = 0 if g < 3 else 2
        row = g if src is None else int(src[g])
        if row >= 7:
            assert np.all(u[g] == 0)
            continue
        written.add(row)
        for c in range(24):
            total = f["base"][row][c]
            for j in range(8):
                low = sum(f["x"][row][k] * f["A"][e][j][k] for k in range(16))
                assert abs(u[g][j] - low) < 1e-12
                total += float(t["scale"][e]) * low * f["B"][e][c][j]
            assert abs(y[row][c] - total) < 1e-11
    assert {i for i in range(7) if not np.isnan(y[i][0])} == written


def test_lora_gradients_against_differences():
    t, counts, src, rng = _case()
    dy = _bits(rng, 7, 24)
    u, _ = P.lora_fwd(t["x"], t["A"], t["B"], t["scale"], counts, 5, src)
    dx, dA, dB, w = P.lora_bwd(dy, t["x"], t["A"], t["B"], t["scale"], counts, 5, u, src)
    d = F.bf16_bits_to_f64(dy)

    def loss(**new):
        v = {k: F.bf16_bits_to_f64(t[k]) for k in ("x", "A", "B")} | new
        total = 0.0
        for e, g, rows in P.lora_rows(counts, 5, src, 7):
            total += np.sum(d[rows] * (float(t["scale"][e]) * ((v["x"][rows] @ v["A"][e].T) @ v["B"][e].T)))
        return total
    for name, grad in (("x", dx), ("A", dA), ("B", dB)):
        v = F.bf16_bits_to_f64(t[name])
        for _ in range(10):
            i = tuple(rng.integers(0, n) for n in v.shape)
            up, down = v.copy(), v.copy()
            up[i] += 1e-3
            down[i] -= 1e-3
            want = (loss(**{name: up}) - loss(**{name: down})) / 2e-3
            got = 0.0 if np.isnan(grad[i]) else grad[i]
            assert abs(got - want) < 1e-7 * max(1.0, abs(want))


def test_counts_are_clipped():
    rows = P.lora_rows([3, -2, 5, 4], 6, None, 100)
    assert [list(g) for _, g, _ in rows] == [[0, 1, 2], [], [3, 4, 5], []]


def test_adamw_closed_forms():
    # the first step from zero states moves every element by lr against its gradient's sign
    g = np.array([3.0, -0.01, 5e3])
    p, m, v = P.adamw(np.ones(3), g, np.zeros(3), np.zeros(3), 0.1, 0.9, 0.999, 0.0, 1)
    assert np.allclose(p, 1 - 0.1 * np.sign(g), atol=1e-12) and np.allclose(m, 0.1 * g) and np.allclose(v, 1e-3 * g * g)
    # without a gradient only the decay is left, and states that were 0 stay
    p, m, v = P.adamw([2.0], [0.0], [0.0], [0.0], 0.1, 0.9, 0.999, 1e-8, 5, weight_decay=0.5)
    assert p[0] == 2.0 * (1 - 0.05) and m[0] == v[0] == 0
    # scaling the gradients scales m, and v by the square
    a, b = (P.adamw([1.0], [2.0], [0.0], [0.0], 0.1, 0.8, 0.9, 1e-8, 2, grad_scale=s) for s in (1.0, 0.5))
    assert math.isclose(a[1][0], 2 * b[1][0]) and math.isclose(a[2][0], 4 * b[2][0])


def test_adamw_against_torch():
    import torch
    rng = np.random.default_rng(1)
    p = torch.nn.Parameter(torch.from_numpy(rng.standard_normal(50)))
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    h, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for step in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.from_numpy(g)
        opt.step()
        h, m, v = P.adamw(h, g, m, v, 3e-3, 0.8, 0.95, 1e-6, step, weight_decay=0.1)
        assert np.allclose(h, p.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_state8_codes_are_the_nearest():
    """Against all codes; the values of the codes themselves come back as those codes."""
    rng = np.random.default_rng(2)
    m, v = rng.standard_normal(300), rng.standard_normal(300) ** 4
    cm, ms, cv, vs = P.state8_encode(m, v)
    for i in range(300):
        b = i // 128
        x = math.sqrt(abs(m[i]) / float(ms[b])) * 127
        best = min(range(128), key=lambda c: (abs(c - x), c))
        assert cm[i] == best * np.sign(m[i])
        x = math.sqrt(math.sqrt(v[i]) / float(vs[b])) * 255
        assert cv[i] == max(1, min(range(256), key=lambda c: (abs(c - x), c)))
    m2, v2 = P.state8_decode(cm, ms, cv, vs)
    again = P.state8_encode(m2, v2)
    assert np.array_equal(again[0], cm) and np.array_equal(again[2], cv)


def test_state8_edges():
    m = np.zeros(256)
    v = np.zeros(256)
    m[3], v[3] = -2.0, 4.0
    v[5], m[5] = 1e-30, 1e-30                    # far below the block's largest: m is lost, v is not
    cm, ms, cv, vs = P.state8_encode(m, v)
    assert cm[3] == -127 and cv[3] == 255 and ms[0] == 2 and vs[0] == 2
    assert cm[5] == 0 and cv[5] == 1 and ms[1] == vs[1] == 0 and not cm[128:].any() and not cv[128:].any()
    m[200] = np.nan
    _, ms, _, vs = P.state8_encode(m, v)
    assert np.isnan(ms[1]) and np.isnan(vs[1]) and ms[0] == 2
    # a tie under the square root goes to the lower code
    m = np.zeros(128)
    m[0], m[1] = 64516.0, 9.0                    # sqrt(9 / 64516) * 127 = 1.5
    assert list(P.state8_encode(m, np.zeros(128))[0][:2]) == [127, 1]


def test_grad_norm():
    assert P.grad_norm([[3.0], [4.0]], 1.0) == (5.0, 1.0 / (5.0 + 1e-6))
    assert P.grad_norm([[3.0], [], [4.0]], 10.0)[1] == 1.0 and P.grad_norm([], 1.0) == (0.0, 1.0)
