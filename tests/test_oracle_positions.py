"""The fp64 oracle of the position operators against independent forms: torch
autograd and central differences for the gradients, hand cases for positions,
buckets and masked rows."""
import math

import numpy as np
import pytest
import torch

import synth
from oracle import attention as A
from oracle import positions as N


def test_positions_restart_at_every_document():
    assert N.positions(synth.cu_from_lengths([3, 1, 2])).tolist() == [0, 1, 2, 0, 0, 1]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_the_complex_product(interleaved):
    rng = np.random.default_rng(0)
    x, f = rng.normal(size=(7, 2, 8)), np.array([1.0, 0.1, 0.01])
    y = N.norm_rope(x, np.array([0, 4, 7]), inv_freq=f, norm=False, interleaved=interleaved)
    a, b = N.pair_dims(6, interleaved)
    p = np.array([0, 1, 2, 3, 0, 1, 2])[:, None, None]
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * p * f)
    assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag) and np.array_equal(y[..., 6:], x[..., 6:])


@pytest.mark.parametrize("norm,interleaved", [(True, False), (True, True), (False, False)])
def test_norm_rope_gradient_against_differences(norm, interleaved):
    rng = np.random.default_rng(1)
    x, dy = rng.normal(size=(5, 3, 16)), rng.normal(size=(5, 3, 16))
    w = rng.normal(size=16) if norm else None
    cu, f = np.array([0, 3, 5]), np.array([1.0, 0.3, 0.1, 0.02])
    kw = dict(inv_freq=f, norm=norm, eps=1e-3, interleaved=interleaved)
    dx, dw = N.norm_rope_bwd(x, dy, cu, w, **kw)

    def loss(x_, w_):
        return (N.norm_rope(x_, cu, w_, **kw) * dy).sum()
    h = 1e-6
    for idx in [(0, 0, 0), (2, 1, 5), (4, 2, 15), (3, 0, 9)]:
        e = np.zeros_like(x)
        e[idx] = h
        assert dx[idx] == pytest.approx((loss(x + e, w) - loss(x - e, w)) / (2 * h), rel=1e-6, abs=1e-8)
    if norm:
        for i in (0, 3, 4, 11, 15):
            e = np.zeros(16)
            e[i] = h
            assert dw[i] == pytest.approx((loss(x, w + e) - loss(x, w - e)) / (2 * h), rel=1e-6, abs=1e-8)


def test_buckets():
    assert N.bucket_of([0, 1, 2, 3, 4, 100], [0, 1, 4, 4]).tolist() == [0, 1, 1, 1, 3, 3]


def test_bias_attention_without_bias_is_the_attention():
    D = [5, 1, 30]
    q, k, v = synth.make_qkv(36, 4, 2, 16, seed=1)
    cu = synth.cu_from_lengths(D)
    o, lse = N.bias_attention(q, k, v, np.zeros((4, 3)), [0, 2, 9], cu)
    o2, l2 = A.attention_per_doc(q, k, v, cu)
    assert np.allclose(o, o2, atol=1e-13) and np.allclose(lse, l2, atol=1e-13)


def test_bias_attention_gradients_against_autograd_and_differences():
    D, hq, hkv, d, starts = [9, 1, 14], 4, 2, 8, [0, 1, 2, 5]
    T = sum(D)
    rng = np.random.default_rng(2)
    q, k, v, do = (rng.normal(size=(T, h, d)) for h in (hq, hkv, hkv, hq))
    b = rng.normal(size=(hq, 4))
    cu = synth.cu_from_lengths(D)
    g = N.bias_attention_bwd(q, k, v, b, starts, do, cu)
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v, b)]
    ids = torch.tensor(A.doc_ids(cu))
    dist = torch.arange(T)[:, None] - torch.arange(T)
    seen = (dist >= 0) & (ids[:, None] == ids)
    bk = torch.bucketize(dist.clamp(min=0), torch.tensor(starts[1:]), right=True)
    kk, vv = (x.repeat_interleave(2, 1) for x in t[1:3])
    s = torch.einsum("ihd,jhd->hij", t[0], kk) / math.sqrt(d) + t[3][:, bk]
    o = torch.einsum("hij,jhd->ihd", torch.softmax(s.masked_fill(~seen, -math.inf), -1), vv)
    assert np.allclose(o.detach().numpy(), N.bias_attention(q, k, v, b, starts, cu)[0], atol=1e-12)
    for a, e in zip(g, torch.autograd.grad((o * torch.tensor(do)).sum(), t)):
        assert np.allclose(a, e.numpy(), atol=1e-12)
    h = 1e-6
    for i in ((0, 0), (1, 2), (3, 3)):
        e = np.zeros_like(b)
        e[i] = h
        up, down = (N.bias_attention(q, k, v, b + x, starts, cu)[0] for x in (e, -e))
        assert g[3][i] == pytest.approx(((up - down) * do).sum() / (2 * h), rel=1e-5, abs=1e-7)


def test_masked_buckets_and_empty_rows():
    """A bias of the type's lowest value or -inf masks its bucket; a row with
    nothing left has O = 0, LSE = -inf and no gradient."""
    q, k, v = synth.make_qkv(6, 2, 2, 8, seed=3)
    cu = synth.cu_from_lengths([1, 5])
    low = np.finfo(np.float32).min
    b = np.array([[low, 0.5], [0.25, -np.inf]])       # head 0: not itself; head 1: only itself
    o, lse = N.bias_attention(q, k, v, b, [0, 1], cu)
    assert np.all(o[[0, 1], 0] == 0) and np.all(lse[0, [0, 1]] == -np.inf) and np.isfinite(lse[0, 2:]).all()
    assert np.allclose(o[:, 1], A.to_f64(v)[:, 1])
    g = N.bias_attention_bwd(q, k, v, b, [0, 1], np.ones((6, 2, 8)), cu)
    assert all(np.isfinite(x).all() for x in g) and g[3][0, 0] == 0 and g[3][1, 1] == 0
    assert np.all(g[0][[0, 1], 0] == 0) and np.all(g[0][:, 1] == 0)
