"""The residual stream between two blocks (fp64 numpy, no shared code with the library), and its gradient with
the norms' Jacobians written out:
  u = y r_y w_post, X = a x + b g(z) u, h = X r w_pre, r of a row v: 1 / sqrt(mean(v^2) + eps).
"""
from __future__ import annotations

import numpy as np


def gate(z, fn):
    """g(z) and g'(z)."""
    if z is None:
        return 1.0, 0.0
    if fn == "plain":
        return z, np.ones_like(z)
    e = np.exp(-np.abs(z))
    g = np.where(z >= 0, 1 / (1 + e), e / (1 + e))
    return g, e / (1 + e) ** 2


def norm_factor(v, eps):
    return 1 / np.sqrt(np.mean(v * v, -1, keepdims=True) + eps)


def forward(x, y=None, z=None, w_post=None, w_pre=None, post_norm=True, gate_fn="sigmoid", a=1.0, b=1.0, eps=1e-6):
    """(X, h)."""
    X = a * x
    if y is not None:
        r = norm_factor(y, eps) if post_norm else 1.0
        X = X + b * gate(z, gate_fn)[0] * (y * r * (1.0 if w_post is None else w_post))
    return X, X * norm_factor(X, eps) * (1.0 if w_pre is None else w_pre)


def backward(dh, dX, X, y=None, z=None, w_post=None, w_pre=None, post_norm=True, gate_fn="sigmoid", a=1.0, b=1.0, eps=1e-6):
    """dict of dx, dy, dgate, dw_post, dw_pre (None where there is none)."""
    D = np.zeros_like(X) if dX is None else dX
    out = dict(dy=None, dgate=None, dw_post=None, dw_pre=None)
    if dh is not None:
        r = norm_factor(X, eps)
        k = dh if w_pre is None else dh * w_pre
        D = D + r * (k - X * r * r * np.mean(k * X, -1, keepdims=True))
        out["dw_pre"] = (dh * X * r).sum(0)
    out["dx"] = a * D
    if y is not None:
        ry = norm_factor(y, eps) if post_norm else 1.0
        w = 1.0 if w_post is None else w_post
        g, dg = gate(z, gate_fn)
        if z is not None:
            out["dgate"] = b * D * (y * ry * w) * dg
        out["dw_post"] = (b * D * g * y * ry).sum(0)
        e = b * D * g * w
        out["dy"] = ry * (e - y * ry * ry * np.mean(e * y, -1, keepdims=True)) if post_norm else e
    return out
