"""A router with biased choices among groups of experts, and the products of sorted rows with
their experts' matrices, in float64 -- the oracle.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

``route_groups`` / ``route_groups_grad``, ``product`` (with its epilogue), ``activation_grad``
and ``product_grad``, each from its definition, token by token and group by group.
"""
from __future__ import annotations

import math

import numpy as np

ACTS = ("none", "relu", "gelu", "silu", "swiglu")


def scores(row: np.ndarray, score: str) -> np.ndarray:
    """The scores of one token's logits (no NaN): a logit of -inf scores 0, logits of +inf share
    a softmax equally, a row of -inf alone scores 0."""
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-row))
    m = row.max()
    if m == -np.inf:
        return np.zeros_like(row)
    e = (row == m).astype(np.float64) if m == np.inf else np.exp(row - m)
    return e / e.sum()


def route_groups(logits, bias, K: int, *, score: str, renorm: bool, n_groups: int = 1, kept: int = 1, group_top: int = 1,
                 scale: float = 1.0):
    """(ids int32 [T, K], weights [T, K])."""
    logits = np.asarray(logits, np.float64)
    logits = np.where(np.isnan(logits), -np.inf, logits)
    T, E = logits.shape
    size = E // n_groups
    ids, w = np.empty((T, K), np.int32), np.empty((T, K))
    for t in range(T):
        s = scores(logits[t], score)
        # without a bias experts are compared by their logits
        c = logits[t].copy() if bias is None else s + np.asarray(bias, np.float64)
        masked = (logits[t] == -np.inf) | np.isnan(c) | (c == -np.inf)
        c[masked] = -np.inf
        value = s if bias is None else c               # what a group sums
        total = []
        for g in range(n_groups):
            live = [(value if group_top == 2 else c)[e] for e in range(g * size, (g + 1) * size) if not masked[e]]
            total.append(sum(sorted(live, reverse=True)[:group_top]) if live else -math.inf)
        groups = sorted(range(n_groups), key=lambda g: (-total[g], g))[:kept]
        order = sorted((e for g in groups for e in range(g * size, (g + 1) * size)), key=lambda e: (-c[e], e))[:K]
        ids[t] = order
        if renorm and score == "softmax":
            p = scores(logits[t][order], "softmax")    # in range however small the chosen scores are
        elif renorm:
            low = min(0.0, logits[t][order].max())
            z = logits[t][order]
            p = np.array([0.0 if v == -np.inf else math.exp(min(v, 0.0) - low) / (1.0 + math.exp(-abs(v))) for v in z])
            p = p / p.sum() if p.sum() > 0 else p
        else:
            p = s[order]
        w[t] = scale * p
    return ids, w


def route_groups_grad(logits, ids, w, d_w, *, score: str, renorm: bool, scale: float = 1.0):
    """d logits [T, E] of the weights w at ids (ids outside the experts contribute nothing)."""
    logits = np.asarray(logits, np.float64)
    logits = np.where(np.isnan(logits), -np.inf, logits)
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        s = scores(logits[t], score)
        pairs = [(int(ids[t, k]), float(w[t, k]), float(d_w[t, k])) for k in range(ids.shape[1]) if 0 <= ids[t, k] < E]
        S = sum(wk * dk for _, wk, dk in pairs)
        if score == "softmax" and not renorm:
            g = np.zeros(E)
            for e, _, dk in pairs:
                g[e] += scale * dk
            out[t] = s * (g - S)
            continue
        for e, wk, dk in pairs:
            d = wk * (dk - S / scale if renorm else dk)
            out[t, e] += d * (1.0 - s[e]) if score == "sigmoid" else d
    return out


def normal_cdf(h: np.ndarray) -> np.ndarray:
    h = np.asarray(h, np.float64)
    return np.array([0.5 * math.erfc(-v / math.sqrt(2.0)) for v in h.reshape(-1)]).reshape(h.shape)


def sigmoid(h: np.ndarray) -> np.ndarray:
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-h))


def activate(h: np.ndarray, act: str) -> np.ndarray:
    if act == "relu":
        return np.where(h <= 0, 0.0, h)                # NaN stays NaN
    if act == "gelu":
        return h * normal_cdf(h)
    if act == "silu":
        return h * sigmoid(h)
    if act == "swiglu":
        half = h.shape[1] // 2
        return activate(h[:, :half], "silu") * h[:, half:]
    return h


def slope(h: np.ndarray, act: str) -> np.ndarray:
    if act == "relu":
        return np.where(np.isnan(h), h, h > 0)
    if act == "gelu":
        return normal_cdf(h) + h * np.exp(-0.5 * h * h) / math.sqrt(2.0 * math.pi)
    if act == "silu":
        s = sigmoid(h)
        return s + h * s * sigmoid(-h)
    return np.ones_like(h)


def runs(offsets, M: int):
    """(group, first row, row behind its last) of each group."""
    ends = [0, M] if offsets is None else [int(v) for v in offsets]
    return [(g, ends[g], ends[g + 1]) for g in range(len(ends) - 1)]


def product(x, w, offsets, bias=None, resid=None, act: str = "none"):
    """(out, h), NaN in rows that no group has."""
    M, N = x.shape[0], w.shape[1]
    h = np.full((M, N), np.nan)
    for g, a, b in runs(offsets, M):
        h[a:b] = x[a:b] @ w[g].T + (0.0 if bias is None else bias[g])
    out = np.full((M, N // 2 if act == "swiglu" else N), np.nan)
    for _, a, b in runs(offsets, M):
        out[a:b] = activate(h[a:b], act) + (0.0 if resid is None else resid[a:b])
    return out, h


def activation_grad(d_out, pre, offsets, N: int, act: str = "none"):
    """(d_pre [M, N], d_bias [G, N]), NaN in rows of d_pre that no group has."""
    M = d_out.shape[0]
    if act == "none":
        d = np.array(d_out, np.float64)
    elif act == "swiglu":
        g, u = pre[:, :N // 2], pre[:, N // 2:]
        d = np.concatenate([d_out * u * slope(g, "silu"), d_out * activate(g, "silu")], axis=1)
    else:
        d = d_out * slope(pre, act)
    out, sums = np.full((M, N), np.nan), []
    for _, a, b in runs(offsets, M):
        out[a:b] = d[a:b]
        sums.append(d[a:b].sum(axis=0))
    return out, np.stack(sums)


def product_grad(d_pre, x, w, offsets):
    """(d_x [M, K], NaN in rows that no group has, d_w [G, N, K])."""
    d_x = np.full((d_pre.shape[0], w.shape[2]), np.nan)
    d_w = np.zeros(w.shape)
    for g, a, b in runs(offsets, d_pre.shape[0]):
        d_x[a:b] = d_pre[a:b] @ w[g]
        d_w[g] = d_pre[a:b].T @ x[a:b]
    return d_x, d_w
