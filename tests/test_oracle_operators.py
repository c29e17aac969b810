"""Pins of the oracle's operators (oracle/operators.py): brute force, closed
forms, the OCP e2m1 table and central differences, all on the CPU."""
import itertools

import numpy as np
import pytest

import workloads as W
from oracle import formats as F
from oracle import operators as P


# ---------------------------------------------------------------- router
def _naive_router(x, k, score, bias, n_groups, topk_groups, group_score, renorm, scale):
    """One token in plain Python, on exact ties as well."""
    import math
    E = len(x)
    if score == "sigmoid":
        s = [1 / (1 + math.exp(-v)) for v in x]
    else:
        m = max(x)
        e = [math.exp(v - m) for v in x]
        s = [v / sum(e) for v in e]
    c = [a + b for a, b in zip(s, bias)] if bias is not None else list(x)
    gc = c if bias is not None or group_score == "max" else s
    size = E // n_groups
    value = []
    for g in range(n_groups):
        top = sorted(gc[g * size:(g + 1) * size], reverse=True)
        value.append(top[0] + top[1] if group_score == "top2" else top[0])
    groups = sorted(range(n_groups), key=lambda g: (-value[g], g))[:topk_groups]
    cand = [e for e in range(E) if e // size in groups]
    ids = sorted(cand, key=lambda e: (-c[e], e))[:k]
    S = sum(s[e] for e in ids) if renorm else 1.0
    return ids, [scale * s[e] / S for e in ids]


@pytest.mark.parametrize("score,group_score", itertools.product(["softmax", "sigmoid"], ["max", "top2"]))
@pytest.mark.parametrize("with_bias,n_groups,renorm", [(False, 1, True), (True, 1, False), (True, 4, True),
                                                       (False, 4, False)])
def test_router_against_plain_python(score, group_score, with_bias, n_groups, renorm):
    rng = np.random.default_rng(7)
    x = np.round(rng.standard_normal((40, 24)) * 2) / 2          # many exact ties
    bias = np.round(rng.standard_normal(24) * 4) / 16 if with_bias else None
    keep = 2 if n_groups > 1 else 1
    ids, w = P.router_topk(x, 5, score, bias, n_groups, keep, group_score, renorm, 2.5)
    for t in range(len(x)):
        rid, rw = _naive_router(list(x[t]), 5, score, bias, n_groups, keep,
                                group_score if n_groups > 1 else "max", renorm, 2.5)
        assert list(ids[t]) == rid
        np.testing.assert_allclose(w[t], rw, rtol=1e-12)


def test_router_special_values():
    inf, nan = np.inf, np.nan
    # a masked row has weights 0 and the lowest ids; masked experts come last
    ids, w = P.router_topk(np.array([[-inf] * 4, [-inf, 1.0, -inf, 0.0]]), 3, "softmax")
    assert ids.tolist() == [[0, 1, 2], [1, 3, 0]] and np.all(w[0] == 0) and w[1, 2] == 0
    np.testing.assert_allclose(w[1, :2], [1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1))])
    # sigmoid scores of -inf are 0: their sum is 0 and so are the weights
    _, w = P.router_topk(np.array([[-inf] * 4]), 2, "sigmoid")
    assert np.all(w == 0)
    # NaN ranks below every number, -0.0 ties with 0.0
    ids, _ = P.router_topk(np.array([[nan, -inf, 2.0, -0.0, 0.0]]), 5, "sigmoid", renorm=False)
    assert ids.tolist() == [[2, 3, 4, 1, 0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_router_gradient_against_differences(score, renorm):
    """Central differences in each logit of L = <dw, w> with the choice held:
    the step h = 1e-5 leaves an error of order h^2 + 1e-16 / h."""
    rng = np.random.default_rng(8)
    x, dw = rng.standard_normal((3, 9)), rng.standard_normal((3, 4))
    ids, _ = P.router_topk(x, 4, score, None, renorm=renorm, scale=1.5)

    def loss(z):
        out = 0.0
        for t in range(3):
            s = P.router_scores(z[t], score)[ids[t]]
            out += np.sum(dw[t] * 1.5 * s / (np.sum(s) if renorm else 1.0))
        return out
    g = P.router_topk_bwd(x, ids, dw, score, renorm, 1.5)
    for t, e in itertools.product(range(3), range(9)):
        d = np.zeros_like(x)
        d[t, e] = 1e-5
        assert abs((loss(x + d) - loss(x - d)) / 2e-5 - g[t, e]) < 1e-8


def test_router_gradient_ids_outside_and_twice():
    x = np.array([[0.3, -0.2, 0.9]])
    one = P.router_topk_bwd(x, np.array([[2, 1]]), np.array([[3.0, 0.5]]), "sigmoid", False)
    two = P.router_topk_bwd(x, np.array([[2, 1, 2, -1, 3]]), np.array([[1.0, 0.5, 2.0, 9.0, 9.0]]), "sigmoid", False)
    np.testing.assert_allclose(one, two)


# ---------------------------------------------------------------- combine
def test_combine_and_gradients():
    rng = np.random.default_rng(9)
    T, k, H, M = 5, 3, 8, 20
    y, d, r = (W.to_bf16_bits(rng.standard_normal(s).astype(np.float32)) for s in ((M, H), (T, H), (T, H)))
    dst = rng.permutation(M)[:T * k].reshape(T, k).astype(np.int32)
    dst[1, 2], dst[3, 0] = -1, M
    w = rng.random((T, k))
    out = P.combine(y, dst, w, r)
    yv = F.bf16_bits_to_f64(y)
    for t in range(T):
        want = F.bf16_bits_to_f64(r)[t].copy()
        for j in range(k):
            if 0 <= dst[t, j] < M:
                want += w[t, j] * yv[dst[t, j]]
        np.testing.assert_allclose(out[t], want, rtol=1e-14)
    dy, named, dw = P.combine_bwd(d, y, dst, w)
    assert named.sum() == T * k - 2 and np.all(dy[~named] == 0) and dw[1, 2] == dw[3, 0] == 0
    # L = <d, out> is linear in w and in y: its differences are the gradients
    dv = F.bf16_bits_to_f64(d)
    base = np.sum(dv * out)
    for t, j in itertools.product(range(T), range(k)):
        w2 = w.copy()
        w2[t, j] += 1.0
        np.testing.assert_allclose(np.sum(dv * P.combine(y, dst, w2, r)) - base, dw[t, j], atol=1e-12)
    np.testing.assert_allclose(np.sum(dy * yv), np.sum(w * dw), rtol=1e-12)


# ---------------------------------------------------------------- norm
def test_rmsnorm_closed_form_and_differences():
    rng = np.random.default_rng(10)
    # a constant row: h = c, rstd = 1 / sqrt(c^2 + eps)
    one = np.full((1, 8), 0x4000, np.uint16)                       # 2.0
    h, rstd, y = P.add_rmsnorm(one, np.full(8, 0x3F80, np.uint16), 0.5, residual_bits=one)
    assert np.all(F.bf16_bits_to_f64(h) == 4.0)
    np.testing.assert_allclose(rstd, 1 / np.sqrt(16.5))
    np.testing.assert_allclose(y, 4 / np.sqrt(16.5))
    hb, dy, dh, wt = (W.to_bf16_bits(rng.standard_normal(s).astype(np.float32)) for s in ((3, 8), (3, 8), (3, 8), (8,)))
    hv, dyv, wv = (F.bf16_bits_to_f64(v) for v in (hb, dy, wt))
    dx, dwt = P.add_rmsnorm_bwd(dy, hb, wt, 1e-5, dh)

    def loss(a, w):
        return np.sum(dyv * a / np.sqrt(np.mean(a * a, axis=1, keepdims=True) + 1e-5) * w)
    for t, i in itertools.product(range(3), range(8)):
        d = np.zeros_like(hv)
        d[t, i] = 1e-5
        num = (loss(hv + d, wv) - loss(hv - d, wv)) / 2e-5 + F.bf16_bits_to_f64(dh)[t, i]
        assert abs(num - dx[t, i]) < 1e-7
    for i in range(8):
        d = np.zeros(8)
        d[i] = 1.0
        assert abs(loss(hv, wv + d) - loss(hv, wv) - dwt[i]) < 1e-12


# ---------------------------------------------------------------- MXFP4
def test_e2m1_table_and_rounding():
    # the OCP e2m1 values
    assert P.e2m1_decode_table().tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    assert P.f64_to_e2m1([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert P.f64_to_e2m1([-0.25, -5.01, 0.26, -0.0]).tolist() == [8, 15, 1, 8]
    t = P.e2m1_decode_table()
    for v in np.linspace(-6, 6, 4801):
        assert abs(t[P.f64_to_e2m1(v)] - v) == np.min(np.abs(t - v))


def test_mxfp4_scale_rule_and_blocks():
    from fractions import Fraction
    rng = np.random.default_rng(11)
    bits = rng.integers(1, 0x7F80, size=400).astype(np.uint16)
    bits[:8] = [0x40C0, 0x40C1, 0x40BF, 0x4100, 0x0001, 0x0080, 0x7F7F, 0x00C0]   # 6, its neighbours, 8, extremes
    for a in F.bf16_bits_to_f64(bits):
        E = int(P.mxfp4_scale_exponent(np.array(a)))
        assert Fraction(a) <= 6 * Fraction(2) ** E
        assert E == -127 or Fraction(a) > 6 * Fraction(2) ** (E - 1)
    v = W.to_bf16_bits((rng.standard_normal((6, 96)) * np.exp2(rng.integers(-20, 20, (6, 1)))).astype(np.float32))
    v[1, 32:64] = 0
    v[2, 5], v[3, 70] = 0x7FC0, 0x7F80                             # a NaN, an infinity
    q, s = P.mxfp4_quantize_rows(v)
    assert q.shape == (6, 48) and s.shape == (6, 3)
    assert s[1, 1] == 0 and s[2, 0] == 255 and s[3, 2] == 255
    assert np.all(q[2, :16] == 0) and np.all(q[3, 32:] == 0)
    d, val = P.mxfp4_dequantize_rows(q, s), F.bf16_bits_to_f64(v)
    ok = np.repeat(s != 255, 32, axis=1)
    X = np.repeat(F.e8m0_value(s), 32, axis=1)
    assert np.all(np.isnan(d[~ok]))
    # half a step: 0.25 below 2, 0.5 below 4, 1 up to 6, in units of the scale
    a = np.abs(val[ok]) / X[ok]
    half = np.where(a <= 2, 0.25, np.where(a <= 4, 0.5, 1.0))
    assert np.all(np.abs(d[ok] - val[ok]) <= half * X[ok])


def test_group_gemm_values_loops():
    rng = np.random.default_rng(12)
    a, b = rng.standard_normal((5, 4)), rng.standard_normal((3, 2, 4))
    out, mag = P.group_gemm_values(a, [2, 0, 3], b)
    for r, e in enumerate([0, 0, 2, 2, 2]):
        for n in range(2):
            assert abs(out[r, n] - sum(a[r, i] * b[e, n, i] for i in range(4))) < 1e-14
            assert abs(mag[r, n] - sum(abs(a[r, i] * b[e, n, i]) for i in range(4))) < 1e-14
