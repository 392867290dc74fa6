"""Plain 64-bit numpy forms of the router, the weighted row movement and the
4-bit expert products, one step of the definition at a time."""

from __future__ import annotations

import numpy as np

NEG = -np.inf


def _scores(logits: np.ndarray, score: str) -> np.ndarray:
    out = np.zeros(logits.shape)
    for t, row in enumerate(logits):
        on = row > NEG                                   # False for NaN too
        if not on.any():
            continue
        if score == "softmax":
            e = np.exp(row[on] - row[on].max())
            out[t, on] = e / e.sum()
        else:
            out[t, on] = 1.0 / (1.0 + np.exp(-row[on]))
    return out


def router(logits: np.ndarray, k: int, score: str = "softmax", bias=None, num_groups: int = 1,
           topk_groups: int = 1, group_top: int = 1, renormalize: bool = True, scale: float = 1.0):
    """(topk_idx [T, k], topk_weights [T, k], probs [T, E]) in 64 bits."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    probs = _scores(logits, score)
    idx = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    per = E // num_groups
    for t in range(T):
        on = logits[t] > NEG
        value = probs[t] + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
        by_value = bias is not None
        if by_value or (num_groups > 1 and group_top > 1):   # values steer: False for NaN
            on = on & (value > NEG)
        rank = value if by_value else logits[t]
        allowed = on.copy()
        if num_groups > 1:
            rating = np.full(num_groups, NEG)
            source = value if by_value or group_top > 1 else logits[t]
            for g in range(num_groups):
                m = on[g * per:(g + 1) * per]
                best = np.sort(source[g * per:(g + 1) * per][m])[::-1][:group_top]
                if best.size:
                    rating[g] = best.sum()
            # stable: ties to the lower group
            keep = np.argsort(-rating, kind="stable")[:topk_groups]
            for g in range(num_groups):
                if g not in keep:
                    allowed[g * per:(g + 1) * per] = False
        order = [e for e in sorted(range(E), key=lambda e: (-rank[e] if allowed[e] else 0.0, e))
                 if allowed[e]][:k]
        idx[t, :len(order)] = order
        w[t, :len(order)] = probs[t, order]
        if renormalize:
            if score == "softmax":                       # without underflow
                l = logits[t, order]
                w[t, :len(order)] = np.exp(l - l.max()) if len(order) else 0.0
            s = w[t].sum()
            if s != 0:                                       # NaN with a logit of +inf
                w[t, :len(order)] /= s
    return idx, w * scale, probs


def router_backward(logits, topk_idx, grad_weights, grad_probs=None, score: str = "softmax",
                    renormalize: bool = True, scale: float = 1.0) -> np.ndarray:
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    p = _scores(logits, score)
    gp = np.zeros((T, E)) if grad_probs is None else np.array(grad_probs, dtype=np.float64)
    gp = np.where(logits > NEG, gp, 0.0)
    direct = np.zeros((T, E))
    for t in range(T):
        at = [j for j, e in enumerate(topk_idx[t]) if 0 <= e < E and logits[t, e] > NEG]
        s = np.array([p[t, topk_idx[t, j]] for j in at])
        g = np.array([grad_weights[t, j] * scale for j in at], dtype=np.float64)
        if renormalize:
            # through the quotient and the score at once: the softmax's own
            # sum cancels, and what is not chosen gets exactly nothing
            r = s / s.sum() if s.sum() > 0 else s
            for j, rj, gj in zip(at, r, g):
                slope = 1.0 if score == "softmax" else 1.0 - p[t, topk_idx[t, j]]
                direct[t, topk_idx[t, j]] += rj * (gj - (r * g).sum()) * slope
        else:
            for j, gj in zip(at, g):
                gp[t, topk_idx[t, j]] += gj
    if score == "softmax":
        # NaN throughout a row with a logit of +inf, its masked experts apart
        return direct + np.where(logits > NEG, p * (gp - (p * gp).sum(1, keepdims=True)), 0.0)
    return direct + p * (1.0 - p) * gp


def permute(x, slot, w, rows: int) -> np.ndarray:
    out = np.zeros((rows, x.shape[1]))
    for t in range(slot.shape[0]):
        for j in range(slot.shape[1]):
            if 0 <= slot[t, j] < rows:
                out[slot[t, j]] = x[t] * (1.0 if w is None else w[t, j])
    return out


def unpermute(y, slot, w) -> np.ndarray:
    T, k = slot.shape
    out = np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= slot[t, j] < y.shape[0]:
                out[t] += y[slot[t, j]] * (1.0 if w is None else w[t, j])
    return out


def pair_dots(tokens, rows, slot):
    """(<tokens[t], rows[slot[t, j]]>, the sum of the products' sizes)."""
    T, k = slot.shape
    d, a = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if 0 <= slot[t, j] < rows.shape[0]:
                d[t, j] = np.dot(tokens[t], rows[slot[t, j]])
                a[t, j] = np.dot(np.abs(tokens[t]), np.abs(rows[slot[t, j]]))
    return d, a


def w4_dequantize(codes, scales, zeros, group: int) -> np.ndarray:
    """[E, N, K] weights in 64 bits; codes uint8 [E, N, K/2]."""
    E, N, half = codes.shape
    q = np.empty((E, N, 2 * half))
    q[:, :, 0::2] = codes & 15
    q[:, :, 1::2] = codes >> 4
    at = np.arange(2 * half) // group
    z = 8.0 if zeros is None else zeros.astype(np.float64)[:, :, at]
    return (q - z) * scales.astype(np.float64)[:, :, at]


def silu(v):
    return v / (1.0 + np.exp(-v))
