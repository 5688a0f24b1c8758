"""float64 restatement of the dense half of a decode step: residual norm with
an 8-bit output, dense product with its epilogue, and sampling.

Test infrastructure only. The definitions are self-defined (the pages describe
none of the three); ``include/qmoe.h`` states them.
"""
from __future__ import annotations

import math

import numpy as np

W_MIN = 2.0 ** -64   # a smaller weight relative to the row's largest counts as none


def quantise(p: np.ndarray, r, group: int):
    """``p`` float64 [T, H] (exact products), ``r`` float64 [T, 1] or 1.0: codes int8 [T, H] and scales
    float64 [T, G]. Zero columns give code 0 and scale 0; columns that are not finite code 0 and scale NaN."""
    T, H = p.shape
    G = H // group if group else 1
    pg = p.reshape(T, G, -1)
    with np.errstate(all="ignore"):
        A = np.abs(pg).max(-1, keepdims=True)
        scales = A[..., 0] * r / 127.0
        good = np.isfinite(A) & np.isfinite(scales[..., None])
        codes = np.where(good & (A > 0), np.rint((pg * 127.0) / A), 0.0)
        scales = np.where(good[..., 0], scales, np.nan)
    return codes.reshape(T, H).astype(np.int8), scales


def norm_q8(x, y, gain, eps: float, group: int):
    """x, y fp32 [T, H] (y may be None), gain fp32 [H] or None -> z fp32, the normalised rows (float64),
    codes int8 and scales float64 [T, G]."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        z = x if y is None else x + np.asarray(y, dtype=np.float32)
        zd = z.astype(np.float64)
        m = (zd * zd).mean(-1, keepdims=True) + eps
        r = np.where(m > 0, 1.0 / np.sqrt(np.where(m > 0, m, 1.0)), 0.0)
        r = np.where(np.isfinite(m), r, np.nan)
        p = zd if gain is None else zd * np.asarray(gain, dtype=np.float32).astype(np.float64)
        norm = p * r
    codes, scales = quantise(p, r, group)
    return z, norm, codes, scales


def act(v: np.ndarray, name: str) -> np.ndarray:
    if name == "relu":
        return np.maximum(v, 0.0)
    if name == "silu":
        return v / (1.0 + np.exp(-v))
    if name == "gelu":
        return v * np.vectorize(lambda t: 0.5 * math.erfc(-t / math.sqrt(2.0)))(v)
    return v


def linear(a, w, a_scale=None, w_scale=None, bias=None, name: str = "none", residual=None):
    """out [M, N] and the sum of |a w| behind every value (for error bounds)."""
    a, w = np.asarray(a, dtype=np.float64), np.asarray(w, dtype=np.float64)
    v, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    if a_scale is not None:
        s = np.asarray(a_scale, dtype=np.float64)[:, None] * np.asarray(w_scale, dtype=np.float64)
        v, mag = v * s, mag * np.abs(s)
    pre = v if bias is None else v + np.asarray(bias, dtype=np.float64)
    out = act(pre, name)
    if residual is not None:
        out = out + np.asarray(residual, dtype=np.float64)
    return out, pre, mag


def sample_row(l, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, u=0.0):
    """(token, prob) of one row of logits (float64 values of fp32 or bf16 numbers)."""
    l = np.asarray(l, dtype=np.float64).copy()
    l[np.isnan(l)] = -np.inf
    order = np.lexsort((np.arange(len(l)), -l))          # logit descending, then the lower index
    m = l[order[0]]
    if m == -np.inf:
        return -1, 0.0
    if temperature == 0:
        return int(order[0]), 1.0
    with np.errstate(all="ignore"):
        w = np.where(l == m, 1.0, np.exp((l - m) / float(temperature)))
    w[np.isnan(w) | (w < W_MIN)] = 0.0
    ws = w[order]
    n = int((ws > 0).sum())
    if 0 < top_k < len(l):
        n = min(n, top_k)
    if min_p > 0:
        n = min(n, int((ws >= float(min_p)).sum()))
    if top_p < 1:
        c = np.cumsum(ws[:n])
        need = max(float(top_p) * c[-1], W_MIN)
        n = min(n, int(np.searchsorted(c, need, side="left")) + 1)
    kept = np.zeros(len(l))
    kept[order[:n]] = ws[:n]
    c = np.cumsum(kept)
    i = int(np.searchsorted(c, float(u) * c[-1], side="right"))
    i = min(i, int(np.nonzero(kept)[0][-1]))
    return i, kept[i] / c[-1]


def sample(logits, temperature=None, top_k=None, top_p=None, min_p=None, u=None):
    T = len(logits)
    got = [sample_row(logits[t], 1.0 if temperature is None else temperature[t], 0 if top_k is None else int(top_k[t]),
                      1.0 if top_p is None else top_p[t], 0.0 if min_p is None else min_p[t], u[t]) for t in range(T)]
    return np.array([g[0] for g in got], dtype=np.int32), np.array([g[1] for g in got])
