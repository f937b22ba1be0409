"""Plain float64 statements of the operators around the MoE layer: residual
addition with RMS norm, MXFP8 rows, the router in the score domain and the MXFP4
projection with low-rank adapters. numpy only; nothing of the package is used."""
from __future__ import annotations

import math

import numpy as np

from .mxfp4_moe_oracle import bf16_bits_to_float, dequant

E4M3_MAX = 448.0


def e4m3_value(code) -> np.ndarray:
    """E4M3 bytes -> float64 (1 sign, 4 exponent bits of bias 7, 3 mantissa bits; 0x7F and 0xFF NaN)."""
    c = np.asarray(code).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * np.exp2(e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def round_e4m3(v) -> np.ndarray:
    """Nearest E4M3 value, ties to even, saturating at +-448 (finite input)."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), E4M3_MAX)
    _, e = np.frexp(a)                          # a = f * 2^e, f in [1/2, 1)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.copysign(np.rint(a / step) * step, v)


def mx8_exponent(amax: float, rule: str) -> int:
    """The shared exponent X of a 32-value block with a finite largest magnitude."""
    if amax == 0:
        return -127
    X = math.frexp(amax)[1] - 1 - 8
    if rule == "nosat" and amax > E4M3_MAX * 2.0 ** X:
        X += 1
    return max(-127, min(127, X))


def mx8_encode(y, rule: str = "ocp"):
    """Rows [T, K] -> (E4M3 values [T, K], scale bytes [T, K/32])."""
    y = np.asarray(y, dtype=np.float64)
    T, K = y.shape
    q = np.zeros((T, K))
    s = np.zeros((T, K // 32), dtype=np.uint8)
    for t in range(T):
        for b in range(K // 32):
            v = y[t, 32 * b:32 * b + 32]
            if not np.all(np.isfinite(v)):
                s[t, b] = 255
                continue
            X = mx8_exponent(float(np.max(np.abs(v))), rule)
            q[t, 32 * b:32 * b + 32] = round_e4m3(v * 2.0 ** -X)
            s[t, b] = X + 127
    return q, s


def mx8_decode(codes, scale) -> np.ndarray:
    f = np.repeat(np.exp2(np.asarray(scale, dtype=np.float64) - 127.0), 32, axis=1)
    return e4m3_value(codes) * np.where(np.repeat(scale, 32, axis=1) == 255, np.nan, f)


def add_rmsnorm(x_bits, gamma_bits, eps: float, residual_bits=None):
    """(h, y) in float64 of bf16 bit rows; h is the sum rounded to float32, as the operator defines it."""
    h = bf16_bits_to_float(x_bits).astype(np.float32)
    if residual_bits is not None:
        h = h + bf16_bits_to_float(residual_bits).astype(np.float32)
    h = h.astype(np.float64)
    rms = np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return h, h / rms * bf16_bits_to_float(gamma_bits).astype(np.float64)


def router_scores(logits, scoring: str) -> np.ndarray:
    """Scores in float64; 0 where the logit is NaN or -inf."""
    x = np.asarray(logits, dtype=np.float64)
    out = np.isnan(x) | (x == -np.inf)
    x = np.where(out, -np.inf, x)
    if scoring == "sigmoid":
        return np.where(out, 0.0, 1.0 / (1.0 + np.exp(-np.where(out, 0.0, x))))
    s = np.zeros_like(x)
    for t, row in enumerate(x):
        m = row.max()
        if m == -np.inf:
            continue
        e = np.where(row == m, 1.0, np.exp(np.where(row == m, 0.0, row - (m if np.isfinite(m) else 0.0))))
        e = np.where((row != m) & (m == np.inf), 0.0, e)
        s[t] = np.where(out[t], 0.0, e) / np.where(out[t], 0.0, e).sum()
    return s


def router_scored(logits, topk: int, scoring: str, bias=None, n_group: int = 1, topk_group: int = 1,
                  group_top: int = 2, renormalise: bool = True, route_scale: float = 1.0):
    """(ids, weights, eligible keys [T, E]: -inf where an expert cannot be chosen)."""
    x = np.asarray(logits, dtype=np.float64)
    s = router_scores(logits, scoring)
    T, E = x.shape
    c = s if bias is None else s + np.asarray(bias, dtype=np.float64)
    ok = ~(np.isnan(x) | (x == -np.inf) | np.isnan(c) | (c == -np.inf))
    key = np.where(ok, x if bias is None else c, -np.inf)
    if n_group > 1:
        gs = E // n_group
        for t in range(T):
            score = []
            for g in range(n_group):
                v = sorted((c[t, e] for e in range(g * gs, (g + 1) * gs) if ok[t, e]), reverse=True)
                score.append(sum(v[:group_top]) if v else -np.inf)
            best = sorted(range(n_group), key=lambda g: (-score[g], g))[:topk_group]
            for g in range(n_group):
                if g not in best or score[g] == -np.inf:
                    key[t, g * gs:(g + 1) * gs] = -np.inf
                    ok[t, g * gs:(g + 1) * gs] = False
    ids = np.full((T, topk), -1, dtype=np.int64)
    w = np.zeros((T, topk))
    for t in range(T):
        order = sorted((e for e in range(E) if ok[t, e]), key=lambda e: (-key[t, e], e))[:topk]
        ids[t, :len(order)] = order
        w[t, :len(order)] = s[t, order]
        if renormalise:
            w[t] = w[t] / w[t].sum() if w[t].sum() > 0 else 0.0
    return ids, w * route_scale, np.where(ok, key, -np.inf)


def linear(x, w, s, ids=None, a_bits=None, b_bits=None, scale=None):
    """(y, magnitude of the main sum, magnitude of the adapter's second sum), x float64 [T, K]."""
    W = dequant(w, s).astype(np.float64)
    y = x @ W.T
    mag = np.abs(x) @ np.abs(W).T
    low = np.zeros_like(y)
    if ids is not None:
        for t, j in enumerate(np.asarray(ids)):
            if 0 <= j < len(a_bits):
                A = bf16_bits_to_float(a_bits[j]).astype(np.float64)
                B = bf16_bits_to_float(b_bits[j]).astype(np.float64)
                v = (A @ x[t]) * (1.0 if scale is None else float(scale[j]))
                y[t] += B @ v
                low[t] = np.abs(B) @ np.abs(v)
    return y, mag, low
