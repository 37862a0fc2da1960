"""The operators around the experts in float64 -- the oracle.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Router (``route`` / ``route_grad``), tokens sorted by expert and back (``sort_pairs``,
``combine`` / ``combine_grad``), e4m3 rounding with one power-of-two scale per 128 values
(``round_rows``) and the product of e4m3 rows with their group's e4m3 matrix
(``scaled_product``), each stated from its definition, with loops where those say it
most plainly.

e4m3: sign, 4 exponent bits with bias 7, 3 mantissa bits; exponent 0 is subnormal
(m * 2^-9), the code 0x7f is NaN and there are no infinities, so 448 is the largest.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes."""
    out = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = np.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[code] = -v if code & 128 else v
    return out


_VALUES = e4m3_values()


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """The nearest e4m3 value of each |v| <= 448 (ties to the even mantissa); NaN stays NaN."""
    v = np.asarray(v, np.float64)
    a = np.abs(np.where(np.isnan(v), 0, v))
    step = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.where(np.isnan(v), np.nan, np.sign(v) * np.round(a / step) * step)


def e4m3_widen(codes: np.ndarray) -> np.ndarray:
    return _VALUES[np.asarray(codes, np.uint8)]


def block_scale(block: np.ndarray) -> float:
    """The smallest power of two s >= 2^-126 with max finite |v| / s <= 448; 1 for zeros."""
    a = np.abs(block[np.isfinite(block)])
    big = float(a.max()) if a.size else 0.0
    if big == 0.0:
        return 1.0
    s = 2.0 ** -126
    while big / s > 448.0:
        s *= 2.0
    return s


def round_rows(x: np.ndarray):
    """(e4m3 values [R, H] in float64, scales [R, ceil(H/128)]) of rows x."""
    x = np.asarray(x, np.float64)
    R, H = x.shape
    out, scales = np.empty_like(x), np.empty((R, -(-H // BLOCK)))
    for r in range(R):
        for b in range(scales.shape[1]):
            part = x[r, b * BLOCK:(b + 1) * BLOCK]
            s = scales[r, b] = block_scale(part)
            out[r, b * BLOCK:(b + 1) * BLOCK] = e4m3_round(np.where(np.isfinite(part), part, np.nan) / s)
    return out, scales


def _terms(z: np.ndarray) -> np.ndarray:
    """exp(z - max) of one row: 0 throughout for a row of -inf, and the limit at +inf."""
    m = z.max()
    if m == -np.inf:
        return np.zeros_like(z)
    with np.errstate(invalid="ignore"):
        return np.where(z == m, 1.0, np.exp(z - m))


def route(logits: np.ndarray, k: int, renorm: bool):
    """(ids [T, k], w [T, k]): the k largest logits, largest first, equal ones ascending;
    NaN as -inf."""
    z = np.array(logits, np.float64)
    z[np.isnan(z)] = -np.inf
    ids = np.empty((z.shape[0], k), np.int32)
    w = np.empty((z.shape[0], k))
    for t, row in enumerate(z):
        ids[t] = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        p = _terms(row)
        total = p[ids[t]].sum() if renorm else p.sum()
        w[t] = p[ids[t]] / total if total > 0 else 0.0
    return ids, w


def route_grad(logits: np.ndarray, ids: np.ndarray, w: np.ndarray, dw: np.ndarray, renorm: bool) -> np.ndarray:
    z = np.array(logits, np.float64)
    z[np.isnan(z)] = -np.inf
    out = np.zeros_like(z)
    for t, row in enumerate(z):
        s = float((w[t] * dw[t]).sum())
        if renorm:
            for e, wk, dk in zip(ids[t], w[t], dw[t]):
                out[t, e] += wk * (dk - s)
        else:
            p = _terms(row)
            p = p / p.sum() if p.sum() > 0 else p
            g = np.zeros_like(row)
            np.add.at(g, ids[t], dw[t])
            out[t] = p * (g - s)
    return out


def sort_pairs(ids: np.ndarray, experts: int):
    """(offsets [experts + 1], rows [T, K]): places of the pairs sorted by (id, token, k)."""
    rows = np.full(ids.shape, -1, np.int32)
    offsets, at = [0], 0
    for e in range(experts):
        for t, k in np.argwhere(ids == e):
            rows[t, k] = at
            at += 1
        offsets.append(at)
    return np.array(offsets, np.int32), rows


def combine(ys: np.ndarray, rows: np.ndarray, w=None, resid=None) -> np.ndarray:
    T, K = rows.shape
    out = np.zeros((T, ys.shape[1])) if resid is None else np.array(resid, np.float64)
    for t in range(T):
        for k in range(K):
            if 0 <= rows[t, k] < T * K:
                out[t] += (1.0 if w is None else float(w[t, k])) * ys[rows[t, k]].astype(np.float64)
    return out


def combine_grad(d_out: np.ndarray, ys: np.ndarray, rows: np.ndarray, w: np.ndarray):
    """(d_ys, with zeros in the rows that no pair has; d_w)."""
    T, K = rows.shape
    d_ys, d_w = np.zeros(ys.shape), np.zeros(rows.shape)
    for t in range(T):
        for k in range(K):
            r = rows[t, k]
            if 0 <= r < T * K:
                d_ys[r] = float(w[t, k]) * d_out[t].astype(np.float64)
                d_w[t, k] = float(d_out[t].astype(np.float64) @ ys[r].astype(np.float64))
    return d_ys, d_w


def widen_rows(values: np.ndarray, scales: np.ndarray) -> np.ndarray:
    return values * np.repeat(scales.astype(np.float64), BLOCK, axis=1)[:, :values.shape[1]]


def widen_matrix(values: np.ndarray, scales: np.ndarray) -> np.ndarray:
    s = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, axis=0), BLOCK, axis=1)
    return values * s[:values.shape[0], :values.shape[1]]


def scaled_product(x: np.ndarray, w, offsets) -> np.ndarray:
    """Rows x (widened) times the matrix w[g] (widened) of their group; NaN in rows of none."""
    out = np.full((x.shape[0], w[0].shape[0]), np.nan)
    for g in range(len(w)):
        out[offsets[g]:offsets[g + 1]] = x[offsets[g]:offsets[g + 1]] @ w[g].T
    return out


def swiglu(h: np.ndarray) -> np.ndarray:
    i = h.shape[1] // 2
    return h[:, :i] / (1.0 + np.exp(-h[:, :i])) * h[:, i:]
