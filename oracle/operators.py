"""Plain CPU oracle of the operators around the expert GEMMs: the router and
its gradient, the combine and its gradients, residual addition + RMS norm and
its gradients, and MXFP4 quantisation and its grouped product.

TEST INFRASTRUCTURE ONLY, like the rest of this package: numpy in float64,
token by token or row by row, no code shared with the GPU path.  [MEGA] §2.1
gives the routing probabilities and the weighted sum of the expert outputs;
the other definitions are those of include/moe_glu.h.
"""
from __future__ import annotations

import math

import numpy as np

from .formats import bf16_bits_to_f64, bf16_round, e8m0_byte, e8m0_value, f64_to_bf16_bits
from .moe import exclusive_offsets


# ============================================================================ router
def router_scores(x: np.ndarray, score: str) -> np.ndarray:
    """Scores of one token's logits; a softmax row of -inf alone has scores 0."""
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        if np.all(x == -np.inf):
            return np.zeros_like(x)
        e = np.exp(x - np.max(x[~np.isnan(x)], initial=-np.inf))
        return e / np.sum(e)


def _order(v: np.ndarray) -> np.ndarray:
    """Indices by value, largest first, ties by index, NaN after every number."""
    nan = np.isnan(v)
    return np.lexsort((np.arange(len(v)), -np.where(nan, 0.0, v), nan))


def router_topk(logits, k, score="softmax", bias=None, n_groups=1, topk_groups=1,
                group_score="max", renorm=True, scale=1.0):
    """ids int32 [T][k] and weights float64 [T][k] (see include/moe_glu.h)."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    ids = np.empty((T, k), dtype=np.int32)
    weights = np.empty((T, k))
    size = E // n_groups
    for t in range(T):
        x = logits[t]
        s = router_scores(x, score)
        choice = x if bias is None else s + np.asarray(bias, dtype=np.float64)
        open_ = np.ones(E, dtype=bool)
        if n_groups > 1:
            value = np.full(n_groups, np.nan)
            for g in range(n_groups):
                v = choice[g * size:(g + 1) * size]
                if group_score == "top2" and bias is None:
                    v = s[g * size:(g + 1) * size]
                v = np.sort(v[~np.isnan(v)])[::-1]
                if group_score == "top2" and len(v) >= 2:
                    value[g] = v[0] + v[1]
                elif group_score == "max" and len(v) >= 1:
                    value[g] = v[0]
            keep = _order(value)[:topk_groups]
            open_ = np.isin(np.arange(E) // size, keep)
        cand = np.flatnonzero(open_)
        ids[t] = cand[_order(choice[cand])[:k]]
        sel = s[ids[t]]
        total = np.sum(sel) if renorm else 1.0
        weights[t] = scale * sel / total if total != 0 else 0.0
    return ids, weights


def router_topk_bwd(logits, ids, dweights, score="softmax", renorm=True, scale=1.0):
    """d(logits) float64 [T][E], by the formulas in include/moe_glu.h."""
    logits = np.asarray(logits, dtype=np.float64)
    dweights = np.asarray(dweights, dtype=np.float64)
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        s = router_scores(logits[t], score)
        sel = [(int(e), g) for e, g in zip(ids[t], dweights[t]) if 0 <= e < E]
        S = sum(s[e] for e, _ in sel) if renorm else 1.0
        if S == 0 or (score == "softmax" and np.all(logits[t] == -np.inf)):
            continue
        dot = sum(g * s[e] for e, g in sel) if renorm else 0.0
        ds = np.zeros(E)
        for e, g in sel:
            ds[e] += scale / S * (g - dot / S)
        if score == "sigmoid":
            out[t] = ds * s * (1.0 - s)
        else:
            out[t] = s * (ds - np.sum(ds * s))
    return out


# ============================================================================ combine
def combine(y_bits, dst, weights, residual_bits=None):
    """float64 [T][H]: residual + sum_j w y[dst] (not rounded)."""
    y = bf16_bits_to_f64(y_bits)
    dst = np.asarray(dst)
    T, k = dst.shape
    out = np.zeros((T, y.shape[1])) if residual_bits is None else bf16_bits_to_f64(residual_bits)
    for t in range(T):
        for j in range(k):
            if 0 <= dst[t, j] < len(y):
                out[t] += (1.0 if weights is None else float(weights[t, j])) * y[dst[t, j]]
    return out


def combine_bwd(dout_bits, y_bits, dst, weights):
    """dy float64 [M_cap][H] (zero where no pair names the row), named [M_cap]
    bool, dweights float64 [T][k]."""
    y, d = bf16_bits_to_f64(y_bits), bf16_bits_to_f64(dout_bits)
    dst = np.asarray(dst)
    T, k = dst.shape
    dy = np.zeros_like(y)
    named = np.zeros(len(y), dtype=bool)
    dw = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = dst[t, j]
            if 0 <= r < len(y):
                dy[r] += (1.0 if weights is None else float(weights[t, j])) * d[t]
                named[r] = True
                dw[t, j] = np.sum(d[t] * y[r])
    return dy, named, dw


# ============================================================================ add + RMS norm
def add_rmsnorm(x_bits, weight_bits, eps, residual_bits=None):
    """h bf16 bits, rstd float64 [T], y float64 [T][H] (not rounded)."""
    x = bf16_bits_to_f64(x_bits)
    if residual_bits is not None:
        x = bf16_round(x + bf16_bits_to_f64(residual_bits))
    rstd = 1.0 / np.sqrt(np.mean(x * x, axis=1) + eps)
    return f64_to_bf16_bits(x), rstd, x * rstd[:, None] * bf16_bits_to_f64(weight_bits)


def add_rmsnorm_bwd(dy_bits, h_bits, weight_bits, eps, dh_bits=None):
    """dx float64 [T][H] (not rounded) and dweight float64 [H]."""
    dy, h, w = (bf16_bits_to_f64(v) for v in (dy_bits, h_bits, weight_bits))
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    n = h * rstd
    g = dy * w
    dx = rstd * (g - n * np.mean(g * n, axis=1, keepdims=True))
    if dh_bits is not None:
        dx = dx + bf16_bits_to_f64(dh_bits)
    return dx, np.sum(dy * n, axis=0)


# ============================================================================ MXFP4
E2M1_MAX = 6.0


def e2m1_decode_table() -> np.ndarray:
    """Values of the 16 e2m1 codes: sign, 2 exponent bits (bias 1), 1 mantissa bit."""
    v = np.empty(16)
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        mag = m * 0.5 if e == 0 else (1.0 + 0.5 * m) * 2.0 ** (e - 1)
        v[c] = -mag if c & 8 else mag
    return v


def f64_to_e2m1(x) -> np.ndarray:
    """Nearest e2m1 code of |x| <= 6, ties to the even code, sign kept."""
    x = np.asarray(x, dtype=np.float64)
    mag = e2m1_decode_table()[:8]
    a = np.abs(x)[..., None]
    d = np.abs(a - mag)
    best = d.min(axis=-1, keepdims=True)
    tie = d == best                       # one code, or two neighbours: the even one
    code = np.where(tie & (np.arange(8) % 2 == 0), 2, tie.astype(int)).argmax(axis=-1)
    return (code + 8 * np.signbit(x)).astype(np.uint8)


def mxfp4_scale_exponent(amax) -> np.ndarray:
    """The smallest E in [-127, 127] with amax / 2^E <= 6 (128: not finite)."""
    amax = np.asarray(amax, dtype=np.float64)
    out = np.full(amax.shape, -127, dtype=np.int64)
    for i, a in np.ndenumerate(amax):
        if not np.isfinite(a):
            out[i] = 128
        elif a > 0:
            E = math.frexp(a)[1] - 4                  # a / 2^E >= 8: too small a scale by one or two
            while a > math.ldexp(E2M1_MAX, E):
                E += 1
            out[i] = min(max(E, -127), 127)
    return out


def mxfp4_quantize_rows(v_bits):
    """bf16 bits [R][C] -> code bytes [R][C/2] (even column in the lower
    nibble) and E8M0 bytes [R][C/32]; a block that is not finite: scale 0xFF,
    zero codes."""
    v = bf16_bits_to_f64(v_bits)
    R, C = v.shape
    b = v.reshape(R, C // 32, 32)
    amax = np.max(np.abs(b), axis=2)                  # NaN if a NaN is in the block
    E = mxfp4_scale_exponent(amax)
    fin = E != 128
    q = f64_to_e2m1(np.where(fin[..., None], b, 0.0) / np.exp2(np.where(fin, E, 0).astype(np.float64))[..., None])
    q = np.where(fin[..., None], q, 0).astype(np.uint8).reshape(R, C)
    return q[:, 0::2] | (q[:, 1::2] << 4), e8m0_byte(E).astype(np.uint8)


def mxfp4_dequantize_rows(q, s) -> np.ndarray:
    """float64 values [..., C] of code bytes [..., C/2] and scales [..., C/32]."""
    q = np.asarray(q)
    t = e2m1_decode_table()
    v = np.stack([t[q & 15], t[q >> 4]], axis=-1).reshape(q.shape[:-1] + (q.shape[-1] * 2,))
    return v * np.repeat(e8m0_value(np.asarray(s)), 32, axis=-1)


def group_gemm_values(a, counts, b):
    """float64 out_e = A_e B_e^T of float64 rows a [M][K] and weights b
    [E][N][K], and sum_k |a b| beside it, over the routed rows."""
    off = exclusive_offsets(counts)
    out = np.zeros((int(off[-1]), b.shape[1]))
    mag = np.zeros_like(out)
    for e in range(len(counts)):
        r = slice(int(off[e]), int(off[e + 1]))
        out[r] = a[r] @ b[e].T
        mag[r] = np.abs(a[r]) @ np.abs(b[e]).T
    return out, mag
