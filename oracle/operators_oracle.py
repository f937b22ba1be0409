"""Plain float64 statements of the operators around the MoE layer: residual
addition with RMS norm, MXFP8 rows, the norms after and before a block with its gate and
their gradient, the router in the score domain with its balance losses and gradients, the
gradient of the combination of routes and the MXFP4 projection with low-rank adapters. numpy only; nothing of the package is used."""
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


def gate_values(gate, act: str):
    """(g, dg / dgate) of gate values of any shape; (1, 0) without a gate."""
    if gate is None:
        return np.ones((1, 1)), np.zeros((1, 1))
    g = np.asarray(gate, dtype=np.float64)
    if act == "linear":
        return g, np.ones_like(g)
    e = np.exp(-np.abs(g))
    s = np.where(g >= 0, 1 / (1 + e), e / (1 + e))
    return s, e / (1 + e) ** 2


def sandwich_norm(x, residual, post_gamma=None, pre_gamma=None, gate=None, act="linear", scale=None, eps=1e-5):
    """dict of n, h, y (None without pre_gamma), r1, r2 [T] (1 where there is no norm), float64."""
    x, residual = np.asarray(x, dtype=np.float64), np.asarray(residual, dtype=np.float64)
    T = x.shape[0]
    r1 = r2 = np.ones(T)
    n = x
    if post_gamma is not None:
        r1 = 1 / np.sqrt(np.mean(x * x, axis=1) + eps)
        n = x * r1[:, None] * post_gamma
    h = (1.0 if scale is None else float(scale)) * residual + gate_values(gate, act)[0] * n
    y = None
    if pre_gamma is not None:
        r2 = 1 / np.sqrt(np.mean(h * h, axis=1) + eps)
        y = h * r2[:, None] * pre_gamma
    return dict(n=n, h=h, y=y, r1=r1, r2=r2)


def sandwich_norm_backward(dh, dy, x, h, r1, r2, post_gamma=None, pre_gamma=None, gate=None, act="linear",
                           residual=None, scale=None):
    """Gradients in float64 from the kept x, h, r1 and r2: dict of x, residual, post_gamma, pre_gamma,
    gate (the full [T, K] terms, not yet summed to the gate's shape) and residual_scale."""
    X = x * r1[:, None] if post_gamma is not None else x
    d = np.zeros_like(x) if dh is None else np.array(dh, dtype=np.float64)
    out = {}
    if pre_gamma is not None:
        out["pre_gamma"] = np.zeros(x.shape[1])
    if dy is not None:
        H = h * r2[:, None]
        v = dy * pre_gamma
        d = d + r2[:, None] * (v - H * np.mean(v * H, axis=1, keepdims=True))
        out["pre_gamma"] = np.sum(dy * H, axis=0)
    a = 1.0 if scale is None else float(scale)
    out["residual"] = a * d
    if residual is not None:
        out["residual_scale"] = np.sum(d * residual)
    g, dg = gate_values(gate, act)
    dn = g * d
    n = X
    if post_gamma is not None:
        u = dn * post_gamma
        out["x"] = r1[:, None] * (u - X * np.mean(u * X, axis=1, keepdims=True))
        out["post_gamma"] = np.sum(dn * X, axis=0)
        n = X * post_gamma
    else:
        out["x"] = dn
    out["gate"] = d * n * dg
    return out


def _masked(logits):
    x = np.asarray(logits, dtype=np.float64)
    return np.where(np.isnan(x), -np.inf, x)


def _counts(most: float, row, scoring: str) -> bool:
    """Whether the router's own fp32 score of the logit `most` of a row is not 0: expf(-x) does not overflow, or a
    softmax's quotient does not vanish. Where the largest score of a sum is 0 there, its quotients are 0, and else
    they are the formula's."""
    if not most > -np.inf:
        return False
    with np.errstate(over="ignore"):
        if scoring == "sigmoid":
            return bool(np.isfinite(np.float32(np.exp(-most))))
        m = row.max()
        if not np.isfinite(m):
            return most == m
        return bool(np.float32(np.float32(np.exp(most - m)) / np.float32(np.sum(np.exp(row - m)))) > 0)


def router_balance(logits, ids, scoring: str, offsets=None):
    """dict of stats [4], counts, prob, slope [S, E] and each token's sequence (-1: not counted)."""
    x, ids = _masked(logits), np.asarray(ids)
    T, E = x.shape
    s = router_scores(x, scoring)
    runs = [(0, T)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))
    S = len(runs)
    counts, prob, slope = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros((S, E))
    seq = np.full(T, -1)
    losses, z = [], []
    for i, (a, b) in enumerate(runs):
        n = 0
        for t in range(max(a, 0), min(b, T)):
            good = [int(e) for e in ids[t] if 0 <= e < E]
            if not good or not np.any(x[t] > -np.inf):
                continue
            n += 1
            seq[t] = i
            for e in good:
                counts[i, e] += 1
            prob[i] += s[t] / s[t].sum() if _counts(x[t].max(), x[t], scoring) else 0.0
            m = x[t].max()
            z.append((m + math.log(np.sum(np.exp(x[t] - m)))) ** 2)
        if n:
            prob[i] /= n
            share = E * counts[i] / counts[i].sum()
            slope[i] = share / n
            losses.append(float(np.sum(share * prob[i])))
    stats = np.array([np.mean(losses) if losses else 0.0, np.mean(z) if z else 0.0, len(z), len(losses)])
    return dict(stats=stats, counts=counts, prob=prob, slope=slope, seq=seq)


def router_weights(logits, ids, scoring: str, renormalise: bool, route_scale: float) -> np.ndarray:
    """The weights of given ids (0 for ids outside [0, E) and for masked experts)."""
    x, ids = _masked(logits), np.asarray(ids)
    s = router_scores(x, scoring)
    w = np.zeros(ids.shape)
    for t in range(ids.shape[0]):
        for j, e in enumerate(ids[t]):
            if 0 <= e < x.shape[1]:
                w[t, j] = s[t, e]
        if renormalise:
            most = max((x[t, e] for e in ids[t] if 0 <= e < x.shape[1]), default=-np.inf)
            w[t] = w[t] / w[t].sum() if _counts(most, x[t], scoring) else 0.0
    return w * route_scale


def router_backward(logits, ids, dw, scoring: str, renormalise: bool, route_scale: float = 1.0, dloss=None,
                    balance=None):
    """(gradient [T, E], sum of the magnitudes of its terms [T, E]) of float64 logits; balance: what
    router_balance returned, for dloss [2]. Token by token through the Jacobian of the scores."""
    x, ids = _masked(logits), np.asarray(ids)
    T, E = x.shape
    s = router_scores(x, scoring)
    # 1 - sigmoid(x) without the cancellation of scores near 1
    rest = router_scores(-x, "sigmoid") if scoring == "sigmoid" else 1 - s
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        good = [(j, int(e)) for j, e in enumerate(ids[t]) if 0 <= e < E and x[t, e] > -np.inf]
        if not any(0 <= e < E for e in ids[t]) or not np.any(x[t] > -np.inf):
            continue
        # ds_a / dx_b and its magnitudes
        if scoring == "sigmoid":
            J = np.diag(s[t] * rest[t])
            Ja = J
        else:
            J = np.diag(s[t]) - np.outer(s[t], s[t])
            Ja = np.diag(s[t]) + np.outer(s[t], s[t])
        if dw is not None:
            g, ga = np.zeros(E), np.zeros(E)
            D = sum(s[t, e] for _, e in good)
            if renormalise and _counts(max((x[t, e] for _, e in good), default=-np.inf), x[t], scoring):
                mean = sum(s[t, e] / D * dw[t, j] for j, e in good)
                amean = sum(s[t, e] / D * abs(dw[t, j]) for j, e in good)
                # q_j (dw_j - mean): through the quotient, whose softmax denominators cancel
                for j, e in good:
                    f = route_scale * s[t, e] / D * (rest[t, e] if scoring == "sigmoid" else 1.0)
                    out[t, e] += f * (dw[t, j] - mean)
                    mag[t, e] += abs(f) * (abs(dw[t, j]) + amean)
            elif not renormalise:
                for j, e in good:
                    g[e] += route_scale * dw[t, j]
                    ga[e] += abs(route_scale * dw[t, j])
                out[t] += g @ J
                mag[t] += ga @ Ja
        if dloss is not None and balance["seq"][t] >= 0:
            slope = balance["slope"][balance["seq"][t]]
            tot = s[t].sum()
            if _counts(x[t].max(), x[t], scoring):
                p = s[t] / tot
                f = p * rest[t] if scoring == "sigmoid" else p
                b = dloss[0] / balance["stats"][3]
                out[t] += b * f * (slope - p @ slope)
                mag[t] += abs(b) * f * (slope + p @ slope)
            m = x[t].max()
            soft = np.exp(x[t] - m)
            lse = m + math.log(soft.sum())
            zt = 2 * dloss[1] * lse * soft / soft.sum() / balance["stats"][2]
            out[t] += zt
            # the logarithm's own error counts beside its value, which may be near 0
            mag[t] += np.abs(zt) + 2 * abs(dloss[1]) * (1 + abs(m)) * soft / soft.sum() / balance["stats"][2]
    return out, mag


def combine_backward(dy, routes, ids=None, weights=None, base: int = 0, experts: int = 0):
    """(dw [T, k], magnitudes [T, k], w_tj dy_t [T, k, K] or None); routes [T, k, K]."""
    T, k, _ = routes.shape
    live = np.ones((T, k), bool)
    if ids is not None:
        i = np.asarray(ids)
        live = (i >= base) & (i < base + experts) if experts else i >= 0
    o = np.where(live[:, :, None], routes, 0.0)
    dw = np.einsum("tk,tjk->tj", dy, o)
    mag = np.einsum("tk,tjk->tj", np.abs(dy), np.abs(o))
    do = None if weights is None else np.where(live[:, :, None], weights[:, :, None] * dy[:, None, :], 0.0)
    return dw, mag, do
