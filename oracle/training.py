"""Plain CPU oracle of the low-rank adapters with their gradients, the AdamW step
with its 8-bit states, and the norm of the gradients.

TEST INFRASTRUCTURE ONLY, like the rest of this package: numpy in float64, group
by group, no code shared with the GPU path.  The definitions are those of
include/moe_glu.h.
"""
from __future__ import annotations

import math

import numpy as np

from .formats import bf16_bits_to_f64


# ============================================================================ adapters
def lora_rows(counts, M_cap, src, T):
    """(group, grouped rows, rows of x and y) for every group, the counts clipped to the capacity and rows whose src
    lies outside left out."""
    out = []
    at = 0
    for e, c in enumerate(np.asarray(counts, dtype=np.int64)):
        n = int(min(max(int(c), 0), M_cap - at))
        g = np.arange(at, at + n)
        r = g if src is None else np.asarray(src, dtype=np.int64)[g]
        ok = (r >= 0) & (r < T)
        out.append((e, g[ok], r[ok]))
        at += n
    return out


def lora_fwd(x, A, B, scale, counts, M_cap, src=None, base=None):
    """float64 values: u [M_cap][r] (NaN in rows that no group holds, 0 where src lies outside), the sum y [T][N] (NaN
    in rows that are not written).  x, A, B, base are bf16 bits."""
    x, A, B = bf16_bits_to_f64(x), bf16_bits_to_f64(A), bf16_bits_to_f64(B)
    T, N, r = len(x), B.shape[1], A.shape[1]
    b = np.zeros((T, N)) if base is None else bf16_bits_to_f64(base)
    u = np.full((M_cap, r), np.nan)
    y = np.full((T, N), np.nan)
    u[:min(M_cap, int(np.maximum(np.asarray(counts, dtype=np.int64), 0).sum()))] = 0.0
    for e, g, rows in lora_rows(counts, M_cap, src, T):
        s = 1.0 if scale is None else float(scale[e])
        u[g] = x[rows] @ A[e].T
        y[rows] = b[rows] + s * (u[g] @ B[e].T)
    return u, y


def lora_bwd(dy, x, A, B, scale, counts, M_cap, u, src=None, dx_base=None):
    """float64 dx [T][K] (NaN in rows that are not written), dA [L][r][K], dB [L][N][r], w [M_cap][r]."""
    dy, x, A, B = (bf16_bits_to_f64(t) for t in (dy, x, A, B))
    T, K = x.shape
    b = np.zeros((T, K)) if dx_base is None else bf16_bits_to_f64(dx_base)
    dx = np.full((T, K), np.nan)
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    w = np.zeros((M_cap, A.shape[1]))
    for e, g, rows in lora_rows(counts, M_cap, src, T):
        s = 1.0 if scale is None else float(scale[e])
        w[g] = dy[rows] @ B[e]
        dx[rows] = b[rows] + s * (w[g] @ A[e])
        dA[e] = s * (w[g].T @ x[rows])
        dB[e] = s * (dy[rows].T @ u[g].astype(np.float64))
    return dx, dA, dB, w


# ============================================================================ AdamW
BLOCK = 128


def state8_decode(cm, m_scale, cv, v_scale):
    """m and v in float64 from 8-bit codes and the blocks' scales."""
    n = len(cm)
    block = np.arange(n) // BLOCK
    cm, cv = cm.astype(np.float64), cv.astype(np.float64)
    m = np.sign(cm) * (cm / 127.0) ** 2 * m_scale.astype(np.float64)[block]
    root = (cv / 255.0) ** 2 * v_scale.astype(np.float64)[block]
    return m, root * root


def _nearest_square(value, scale, top, least):
    """The c with (c / top)^2 scale nearest to value under the square root, the lower of two as near."""
    best, dist = 0, math.inf
    at = math.sqrt(value / scale) * top
    for c in range(max(0, int(at) - 2), min(top, int(at) + 2) + 1):
        d = abs(c - at)
        if d < dist:
            best, dist = c, d
    return max(best, least) if value > 0 else 0


def state8_encode(m, v, scales=None):
    """(cm int8, m_scale fp32, cv uint8, v_scale fp32) of float64 states; ``scales``: the two to take, in the place of
    the roundings of the blocks' largest values."""
    n = len(m)
    blocks = (n + BLOCK - 1) // BLOCK
    cm, cv = np.zeros(n, dtype=np.int8), np.zeros(n, dtype=np.uint8)
    ms, vs = np.zeros(blocks, dtype=np.float32), np.zeros(blocks, dtype=np.float32)
    for b in range(blocks):
        s = slice(b * BLOCK, min(n, (b + 1) * BLOCK))
        with np.errstate(over="ignore", invalid="ignore"):
            root = np.sqrt(v[s])
            ok = np.all(np.isfinite(m[s].astype(np.float32))) and np.all(np.isfinite(root.astype(np.float32)))
        if not ok:
            ms[b] = vs[b] = np.nan
            continue
        ms[b], vs[b] = (np.max(np.abs(m[s])), np.max(root)) if scales is None else (scales[0][b], scales[1][b])
        for i in range(s.start, s.stop):
            if ms[b] > 0:
                cm[i] = int(np.sign(m[i])) * _nearest_square(abs(m[i]), float(ms[b]), 127, 0)
            if vs[b] > 0:
                cv[i] = _nearest_square(math.sqrt(v[i]), float(vs[b]), 255, 1)
    return cm, ms, cv, vs


def adamw(p, g, m, v, lr, beta1, beta2, eps, step, weight_decay=0.0, grad_scale=1.0):
    """p, m, v after one step, in float64."""
    p, g, m, v = (np.asarray(t, dtype=np.float64) for t in (p, g, m, v))
    g = g * float(grad_scale)
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    update = (m / (1.0 - beta1 ** step)) / (np.sqrt(v / (1.0 - beta2 ** step)) + eps)
    return p * (1.0 - lr * weight_decay) - lr * update, m, v


def grad_norm(grads, max_norm):
    """(norm, clip factor) of a list of arrays, by exact summation."""
    norm = math.sqrt(math.fsum(float(x) * float(x) for g in grads for x in np.asarray(g, dtype=np.float64).ravel()))
    return norm, min(1.0, max_norm / (norm + 1e-6))
