"""fp64 oracle of the position operators of document-masked attention.

TEST INFRASTRUCTURE ONLY. Written from the definitions, in numpy:

  head norm and rotation   n = x / sqrt(mean(x^2) + eps) * w; pair i of the
                           leading 2 * len(inv_freq) dimensions of n turned by
                           (token - its document's start) * inv_freq[i]
  their gradient           with the norm's Jacobian written out as a matrix
  bucketed distance bias   s_ij = scale <q_i, k_j> + b[h, bucket(i - j)]
                           inside the intra-document causal mask
"""
from __future__ import annotations

import math

import numpy as np

from .attention import default_scale, doc_ids, to_f64


def positions(cu) -> np.ndarray:
    """Index of every token inside its document."""
    cu = np.asarray(cu, dtype=np.int64)
    return np.arange(int(cu[-1])) - cu[:-1][doc_ids(cu)]


def pair_dims(rot: int, interleaved: bool):
    """The two dimensions of each rotated pair."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotation(pos: int, inv_freq, d: int, interleaved: bool) -> np.ndarray:
    """R(pos) as a d x d matrix."""
    R = np.eye(d)
    f = to_f64(inv_freq) if inv_freq is not None else np.zeros(0)
    for i, (a, b) in enumerate(zip(*pair_dims(2 * len(f), interleaved))):
        t = pos * f[i]
        R[a, a], R[a, b], R[b, a], R[b, b] = math.cos(t), -math.sin(t), math.sin(t), math.cos(t)
    return R


def norm_rope(x, cu, w=None, inv_freq=None, norm=True, eps=1e-6, interleaved=False) -> np.ndarray:
    """x [T][heads][d] -> y."""
    x = to_f64(x)
    if norm:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else to_f64(w))
    pos = positions(cu)
    R = np.stack([rotation(p, inv_freq, x.shape[-1], interleaved) for p in range(pos.max() + 1)])
    return np.einsum("tij,thj->thi", R[pos], x)


def norm_rope_bwd(x, dy, cu, w=None, inv_freq=None, norm=True, eps=1e-6, interleaved=False):
    """(dx, dw) for an upstream dy."""
    x, dy = to_f64(x), to_f64(dy)
    d = x.shape[-1]
    pos = positions(cu)
    R = np.stack([rotation(p, inv_freq, d, interleaved) for p in range(pos.max() + 1)])
    z = np.einsum("tji,thj->thi", R[pos], dy)
    if not norm:
        return z, None
    ww = np.ones(d) if w is None else to_f64(w)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = z * ww
    # d(x r)_i / dx_j = r delta_ij - r^3 x_i x_j / d
    dx = r * g - r ** 3 * x * (g * x).sum(-1, keepdims=True) / d
    return dx, (z * x * r).sum((0, 1))


def bucket_of(distance, starts) -> np.ndarray:
    """Last bucket that starts at or before the distance (distances >= 0)."""
    return (np.asarray(distance)[..., None] >= np.asarray(starts)).sum(-1) - 1


def _scores(q, k, b, starts, scale):
    """Scores of one document and head, -inf where masked; distances."""
    n = len(q)
    dist = np.arange(n)[:, None] - np.arange(n)
    s = scale * (q @ k.T) + b[bucket_of(np.maximum(dist, 0), starts)]
    return np.where(dist >= 0, s, -np.inf), dist


def bias_attention(q, k, v, bias, starts, cu, scale=None, key_block=None):
    """(O, LSE) of document-masked attention with bias[h, bucket(i - j)] added to
    the scores; a bias of -1e6 or less masks its bucket. Rows with no key left
    get O = 0, LSE = -inf. key_block (lo, hi) restricts the keys."""
    q, k, v, bias = to_f64(q), to_f64(k), to_f64(v), to_f64(bias)
    bias = np.where(bias <= -1e6, -np.inf, bias)
    T, hq, d = q.shape
    G = hq // k.shape[1]
    scale = default_scale(d) if scale is None else scale
    o, lse = np.zeros((T, hq, d)), np.full((hq, T), -np.inf)
    lo, hi = (0, T) if key_block is None else key_block
    for a, e in zip(cu[:-1], cu[1:]):
        for h in range(hq):
            s, _ = _scores(q[a:e, h], k[a:e, h // G], bias[h], starts, scale)
            outside = (np.arange(a, e) < lo) | (np.arange(a, e) >= hi)
            s[:, outside] = -np.inf
            m = s.max(1)
            seen = np.isfinite(m)
            p = np.exp(s - np.where(seen, m, 0.0)[:, None])
            l = p.sum(1)
            o[a:e, h] = np.where(seen[:, None], p @ v[a:e, h // G] / np.where(seen, l, 1.0)[:, None], 0.0)
            with np.errstate(divide="ignore"):
                lse[h, a:e] = np.where(seen, m + np.log(np.where(seen, l, 1.0)), -np.inf)
    return o, lse


def bias_attention_bwd(q, k, v, bias, starts, do, cu, scale=None):
    """(dQ, dK, dV, dbias) of bias_attention for an upstream dO."""
    o, lse = bias_attention(q, k, v, bias, starts, cu, scale)
    q, k, v, bias, do = to_f64(q), to_f64(k), to_f64(v), to_f64(bias), to_f64(do)
    bias = np.where(bias <= -1e6, -np.inf, bias)
    T, hq, d = q.shape
    G = hq // k.shape[1]
    scale = default_scale(d) if scale is None else scale
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    db = np.zeros((hq, len(starts)))
    for a, e in zip(cu[:-1], cu[1:]):
        for h in range(hq):
            g = h // G
            s, dist = _scores(q[a:e, h], k[a:e, g], bias[h], starts, scale)
            l = lse[h, a:e]
            p = np.where(np.isfinite(l)[:, None], np.exp(s - np.where(np.isfinite(l), l, 0.0)[:, None]), 0.0)
            dp = do[a:e, h] @ v[a:e, g].T
            ds = p * (dp - (do[a:e, h] * o[a:e, h]).sum(1, keepdims=True))
            dq[a:e, h] = scale * ds @ k[a:e, g]
            dk[a:e, g] += scale * ds.T @ q[a:e, h]
            dv[a:e, g] += p.T @ do[a:e, h]
            np.add.at(db[h], bucket_of(np.maximum(dist, 0), starts)[dist >= 0], ds[dist >= 0])
    return dq, dk, dv, db
