"""Attention under a sliding window with sinks, and what a shard needs for it,
from the definition (fp64 numpy, no shared code with the library): query i of a
document that starts at o sees key j <= i if i - j < window or j - o < sinks.
"""
from __future__ import annotations

import math

import numpy as np

from . import attention as A


def visible(n: int, window: int, sinks: int) -> np.ndarray:
    """[n][n] of one document: row i's keys."""
    dist = np.arange(n)[:, None] - np.arange(n)
    return (dist >= 0) & ((dist < window) | (np.arange(n) < sinks))


def needed_keys(doclens, pieces, window: int, sinks: int) -> np.ndarray:
    """Flags of the packed sequence's keys that the queries of `pieces`, (doc,
    start, end) in global rows, see."""
    off = np.concatenate([[0], np.cumsum(doclens)])
    need = np.zeros(off[-1], bool)
    for doc, a, b in pieces:
        o, e = off[doc], off[doc + 1]
        need[o:e] |= visible(e - o, window, sinks)[a - o:b - o].any(0)
    return need


def pairs(doclens, pieces, window: int, sinks: int) -> int:
    off = np.concatenate([[0], np.cumsum(doclens)])
    return sum(int(visible(doclens[doc], window, sinks)[a - off[doc]:b - off[doc]].sum()) for doc, a, b in pieces)


def attention(q, k, v, doclens, window: int, sinks: int, scale: float | None = None, kv_block=None):
    """(O [T][hq][d], LSE [hq][T]); a row without a key in the block: 0 and -inf."""
    q, k, v = (A.to_f64(x) for x in (q, k, v))
    T, hq, d = q.shape
    G, scale = hq // k.shape[1], scale or 1 / math.sqrt(d)
    lo, hi = kv_block or (0, T)
    out, lse = np.zeros_like(q), np.full((hq, T), -np.inf)
    a = 0
    for n in doclens:
        key = np.arange(a, a + n)
        seen = visible(n, window, sinks) & (key >= lo) & (key < hi)
        for h in range(hq):
            s = np.where(seen, scale * q[a:a + n, h] @ k[a:a + n, h // G].T, -np.inf)
            m = np.max(s, 1, keepdims=True)
            p = np.exp(s - np.where(np.isfinite(m), m, 0))
            total = p.sum(1, keepdims=True)
            out[a:a + n, h] = p / np.where(total > 0, total, 1) @ v[a:a + n, h // G]
            with np.errstate(divide="ignore"):
                lse[h, a:a + n] = (np.where(np.isfinite(m), m, 0) + np.log(total))[:, 0]
        a += n
    return out, lse


def attention_bwd(q, k, v, do, doclens, window: int, sinks: int, scale: float | None = None):
    """(dQ, dK, dV) of sum(O dO), over the whole window."""
    q, k, v, do = (A.to_f64(x) for x in (q, k, v, do))
    G, scale = q.shape[1] // k.shape[1], scale or 1 / math.sqrt(q.shape[2])
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    a = 0
    for n in doclens:
        e, seen = a + n, visible(n, window, sinks)
        for h in range(q.shape[1]):
            Q, K, V, dO = q[a:e, h], k[a:e, h // G], v[a:e, h // G], do[a:e, h]
            s = np.where(seen, scale * Q @ K.T, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            dp = dO @ V.T
            ds = p * (dp - (p * dp).sum(1, keepdims=True))
            dq[a:e, h] = scale * ds @ K
            dk[a:e, h // G] += scale * ds.T @ Q
            dv[a:e, h // G] += p.T @ dO
        a = e
    return dq, dk, dv
