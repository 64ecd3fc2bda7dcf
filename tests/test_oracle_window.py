"""Pins of the windowed attention's oracle: torch's softmax and autograd in fp64
under a mask written out pair by pair, central differences, windows that cut
nothing, and hand cases."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import window as W

torch = pytest.importorskip("torch")


def inputs(docs, hq, hkv, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    T = sum(docs)
    return [torch.randn(T, h, d, generator=g, dtype=torch.float64) for h in (hq, hkv, hkv, hq)]


def test_hand_cases():
    assert W.visible(5, 2, 1).astype(int).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 1, 1, 0, 0], [1, 0, 1, 1, 0],
                                                       [1, 0, 0, 1, 1]]
    assert W.visible(3, 1, 0).astype(int).tolist() == np.eye(3, dtype=int).tolist()
    assert W.needed_keys([4, 6], [(1, 8, 10)], 2, 1).tolist() == [False] * 4 + [True, False, False, True, True, True]
    assert W.pairs([4, 6], [(0, 0, 4), (1, 8, 10)], 2, 1) == 1 + 2 + 3 + 3 + 3 + 3


@pytest.mark.parametrize("docs,hq,hkv,window,sinks", [([7, 1, 20], 4, 2, 5, 2), ([30], 3, 1, 1, 1), ([11, 12], 2, 2, 100, 3),
                                                       ([25, 2], 2, 1, 8, 0)])
def test_against_autograd_and_differences(docs, hq, hkv, window, sinks):
    q, k, v, do = inputs(docs, hq, hkv, 8)
    T, G = sum(docs), hq // hkv
    seen = torch.zeros(T, T, dtype=torch.bool)
    start = np.repeat(np.concatenate([[0], np.cumsum(docs)[:-1]]), docs)
    for i in range(T):
        for j in range(start[i], i + 1):
            seen[i, j] = bool(i - j < window or j - start[i] < sinks)
    x = [t.clone().requires_grad_() for t in (q, k, v)]
    s = torch.einsum("ihd,jhd->hij", x[0], x[1].repeat_interleave(G, 1)) / 8 ** 0.5
    s = s.masked_fill(~seen, -torch.inf)
    o = torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), x[2].repeat_interleave(G, 1))
    grads = torch.autograd.grad((o * do).sum(), x)
    out, lse = W.attention(q, k, v, docs, window, sinks)
    np.testing.assert_allclose(out, o.detach().numpy(), atol=1e-12)
    np.testing.assert_allclose(lse, torch.logsumexp(s, -1).detach().numpy(), atol=1e-12)
    got = W.attention_bwd(q, k, v, do, docs, window, sinks)
    for a, b in zip(got, grads):
        np.testing.assert_allclose(a, b.numpy(), atol=1e-12)
    arrays, rng = [t.numpy() for t in (q, k, v)], np.random.default_rng(0)
    for which in range(3):
        for _ in range(3):
            at = tuple(int(rng.integers(n)) for n in arrays[which].shape)
            vals = []
            for h in (1e-5, -1e-5):
                y = [a.copy() for a in arrays]
                y[which][at] += h
                vals.append((W.attention(*y, docs, window, sinks)[0] * do.numpy()).sum())
            assert abs((vals[0] - vals[1]) / 2e-5 - got[which][at]) < 1e-7


def test_a_wide_window_is_the_attention():
    docs = [13, 1, 40]
    q, k, v, _ = inputs(docs, 4, 2, 8)
    out, lse = W.attention(q, k, v, docs, 40, 5)
    ref, ref_lse = A.attention_per_doc(q, k, v, np.concatenate([[0], np.cumsum(docs)]))
    np.testing.assert_allclose(out, ref, atol=1e-12)
    np.testing.assert_allclose(lse, ref_lse, atol=1e-12)


def test_blocks_merge():
    docs = [13, 1, 40]
    q, k, v, _ = inputs(docs, 4, 2, 8)
    out, lse = W.attention(q, k, v, docs, 6, 2)
    parts = [W.attention(q, k, v, docs, 6, 2, kv_block=b) for b in ((0, 9), (9, 31), (31, 54))]
    w = np.exp(np.stack([p[1] for p in parts]) - lse)
    np.testing.assert_allclose(sum(x.T[..., None] * p[0] for x, p in zip(w, parts)), out, atol=1e-12)
