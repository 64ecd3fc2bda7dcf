"""Head norm and rotation on the GPU against the definition in 64 bits.

Bounds. With u = 2^-24 (fp32's half step) and the bf16 half step 2^-8, both
relative: a head's mean square takes 16 products and sums in a lane and three
or two more across lanes (19u, half of it in the root), the reciprocal root and
the two factors 4u, the angle 2^-25 pi and its sine and cosine 4u together, the
turned pair 3u: under 32u of the pair's |a| + |b|, then one rounding to bf16.
The gradient has the same parts once more in the projection term: under 64u of
r (|g| + |x| r^2 mean|g x|). The weight gradients add at most 64 rows and heads
in a lane and then 3 + 3 + 4 + 4 + 2 levels and groups: under 128u of
sum |z x r|."""
import numpy as np
import pytest
import torch

import synth
from oracle import attention as A
from oracle import positions as N

pytestmark = pytest.mark.gpu

U, BF16 = 2.0 ** -24, 2.0 ** -8


def pair_size(x, rot, interleaved):
    """|a| + |b| of the pair that each dimension belongs to (|x| where it does not turn)."""
    m = np.abs(x)
    a, b = N.pair_dims(rot, interleaved)
    out = m.copy()
    out[..., a] = out[..., b] = m[..., a] + m[..., b]
    return out


def make(docs, hq, hkv, d, rot, seed, w_dtype=torch.float32, theta=1e4, spread=1.0):
    T = sum(docs)
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    qkv = (n(T, hq + 2 * hkv, d) * spread).to(torch.bfloat16)
    w = [(1 + 0.2 * n(d)).to(w_dtype) for _ in range(2)]
    f = (theta ** (-torch.arange(0, rot, 2).double() / max(rot, 1))).float() if rot else None
    grads = [n(T, h, d) for h in (hq, hkv, hkv)]
    return qkv, w, f, grads


def session(docs, cp, hq, hkv, d, policy="perdoc"):
    from context_document_masked_gb300.session import CPAttention
    return CPAttention(docs, cp, policy, hq, hkv, d)


def slices(x, hq, hkv):
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]


def check_forward(got, x, docs, w, f, norm, eps, interleaved):
    cu = synth.cu_from_lengths(docs)
    want = N.norm_rope(x, cu, w, f, norm, eps, interleaved)
    flat = N.norm_rope(x, cu, w, None, norm, eps)
    rot = 0 if f is None else 2 * len(f)
    bound = BF16 * np.abs(want) + 32 * U * pair_size(flat, rot, interleaved) + 1e-38
    assert (np.abs(A.to_f64(got) - want) <= bound).all()


def check_backward(got, gw, x, dy, docs, w, f, norm, eps, interleaved):
    cu = synth.cu_from_lengths(docs)
    dx, dw = N.norm_rope_bwd(x, dy, cu, w, f, norm, eps, interleaved)
    rot = 0 if f is None else 2 * len(f)
    x64, size = A.to_f64(x), pair_size(A.to_f64(dy), rot, interleaved)
    if norm:
        ww = np.ones(x64.shape[-1]) if w is None else np.abs(A.to_f64(w))
        r = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + eps)
        g = size * ww
        err = 64 * U * r * (g + np.abs(x64) * r ** 2 * (g * np.abs(x64)).mean(-1, keepdims=True))
    else:
        err = 32 * U * size
    assert (np.abs(A.to_f64(got) - dx) <= BF16 * np.abs(dx) + err + 1e-38).all()
    if gw is not None:
        # 128u of the sums and 32u of z itself
        assert (np.abs(A.to_f64(gw) - dw) <= 160 * U * (size * np.abs(x64) * r).sum((0, 1)) + 1e-38).all()


CASES = [
    # documents, cp, hq, hkv, d, rot, interleaved, norm, weight type
    ([1], 1, 1, 1, 64, 64, False, True, torch.float32),
    ([1, 1, 1], 1, 5, 5, 64, 16, True, True, torch.float32),
    ([7, 1, 130, 128, 129, 3], 2, 4, 2, 128, 128, False, True, torch.float32),
    ([7, 1, 130, 128, 129, 3], 3, 6, 2, 128, 64, True, True, torch.bfloat16),
    ([300, 211], 4, 8, 1, 64, 48, False, True, torch.bfloat16),
    ([300, 211], 1, 12, 12, 64, 64, True, False, None),
    ([257], 2, 9, 3, 128, 0, False, True, None),
    ([40] * 9, 3, 33, 11, 128, 112, False, True, torch.float32),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{len(c[0])}docs_h{c[2]}kv{c[3]}_d{c[4]}_rot{c[5]}" for c in CASES])
def test_forward_and_gradient(cuda, case):
    docs, cp, hq, hkv, d, rot, inter, norm, wt = case
    eps = 1e-5
    qkv, w, f, (dq, dk, dv) = make(docs, hq, hkv, d, rot, seed=len(docs) + hq, w_dtype=wt or torch.float32)
    wq, wk = w if norm and wt else (None, None)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    s = session(docs, cp, hq, hkv, d)
    x = qkv.cuda()
    kw = dict(wq=dev(wq), wk=dev(wk), inv_freq=dev(f), norm=norm, eps=eps, interleaved=inter)
    q, k, v = s.qk_norm_rope(*slices(x, hq, hkv), **kw)
    out = torch.full_like(x, float("nan"))
    parts = slices(out, hq, hkv)
    gw = [torch.zeros(d, device="cuda") for _ in range(2)] if norm else [None, None]
    s.qk_norm_rope_backward(dev(dq), dev(dk), dev(dv), *slices(x, hq, hkv)[:2], **kw, dq_in=parts[0], dk_in=parts[1],
                            dv_in=parts[2], dwq=gw[0], dwk=gw[1])
    torch.cuda.synchronize()
    xq, xk, xv = slices(qkv, hq, hkv)
    check_forward(q, xq, docs, wq, f, norm, eps, inter)
    check_forward(k, xk, docs, wk, f, norm, eps, inter)
    assert torch.equal(v.cpu(), xv)
    check_backward(parts[0], gw[0], xq, dq, docs, wq, f, norm, eps, inter)
    check_backward(parts[1], gw[1], xk, dk, docs, wk, f, norm, eps, inter)
    assert torch.equal(parts[2].cpu(), dv.to(torch.bfloat16))
    assert s.device_status() == 0


def test_no_eps_and_lanes_without_a_head(cuda):
    """eps = 0 with head counts that leave lanes without a head: the gradients
    of the weights are those of the heads alone."""
    docs, hq, hkv, d = [33], 6, 3, 64
    qkv, w, f, (dq, dk, _) = make(docs, hq, hkv, d, d, seed=12)
    s = session(docs, 1, hq, hkv, d)
    x = qkv.cuda()
    gq, gk, _, gwq, gwk = s.qk_norm_rope_backward(dq.cuda(), dk.cuda(), None, *slices(x, hq, hkv)[:2], wq=w[0].cuda(),
                                                  wk=w[1].cuda(), inv_freq=f.cuda(), eps=0.0)
    xq, xk, _ = slices(qkv, hq, hkv)
    check_backward(gq, gwq, xq, dq, docs, w[0], f, True, 0.0, False)
    check_backward(gk, gwk, xk, dk, docs, w[1], f, True, 0.0, False)


def test_far_positions(cuda):
    """Rows at the end of a document of 300,000 tokens, every 10,007th before:
    the angle there is 300,000 inv_freq, and must be as exact as at row 1."""
    T, hq, hkv, d = 300_001, 1, 1, 64
    qkv, w, f, _ = make([T], hq, hkv, d, d, seed=4)
    x = qkv.cuda()
    s = session([T], 1, hq, hkv, d)
    q, k, _ = s.qk_norm_rope(x[:, :1], x[:, 1:2], None, wq=w[0].cuda(), wk=w[1].cuda(), inv_freq=f.cuda(), eps=1e-6)
    rows = list(range(0, T, 10_007)) + [T - 1]
    for got, xx, ww in ((q, qkv[:, 0], w[0]), (k, qkv[:, 1], w[1])):
        xx = A.to_f64(xx[rows])
        n = xx / np.sqrt((xx ** 2).mean(-1, keepdims=True) + 1e-6) * A.to_f64(ww)
        t = np.array(rows)[:, None] * A.to_f64(f)
        want = np.concatenate([n[:, :32] * np.cos(t) - n[:, 32:] * np.sin(t), n[:, :32] * np.sin(t) + n[:, 32:] * np.cos(t)], 1)
        # numpy's own angle is off by half a step of 64 bits of 3e5: 2^-35
        bound = BF16 * np.abs(want) + 32 * U * pair_size(n, 64, False)
        assert (np.abs(A.to_f64(got[rows, 0]) - want) <= bound).all()


@pytest.mark.parametrize("policy", ["llama3", "hybrid", "perdoc"])
def test_shards_make_up_the_whole(cuda, policy):
    """Shard by shard (each writes its own rows alone) and all at once: the
    same bits; the weight gradients add up."""
    docs, cp, hq, hkv, d = [900, 20, 1, 104, 1023], 4, 6, 2, 128
    qkv, w, f, (dq, dk, dv) = make(docs, hq, hkv, d, d, seed=8)
    x, f = qkv.cuda(), f.cuda()
    wq, wk = (t.cuda() for t in w)
    g = [t.cuda() for t in (dq, dk, dv)]
    s = session(docs, cp, hq, hkv, d, policy)
    kw = dict(wq=wq, wk=wk, inv_freq=f)
    whole = s.qk_norm_rope(*slices(x, hq, hkv), **kw)
    gwhole = s.qk_norm_rope_backward(*g, *slices(x, hq, hkv)[:2], **kw)
    nan = float("nan")
    part = [torch.full_like(t, nan) for t in whole]
    gpart = [torch.full_like(t, nan) for t in gwhole[:3]] + [torch.zeros_like(t) for t in gwhole[3:]]
    for j in range(cp):
        before = [t.clone() for t in part]
        s.qk_norm_rope(*slices(x, hq, hkv), **kw, shard=j, q=part[0], k=part[1], v=part[2])
        s.qk_norm_rope_backward(*g, *slices(x, hq, hkv)[:2], **kw, shard=j, dq_in=gpart[0], dk_in=gpart[1], dv_in=gpart[2],
                                dwq=gpart[3], dwk=gpart[4])
        other = torch.ones(sum(docs), dtype=torch.bool)
        other[torch.from_numpy(s.plan.query_indices(j)).long()] = False
        other = other.cuda()
        for a, b in zip(before, part):
            assert torch.equal(a[other].view(torch.int16), b[other].view(torch.int16))
    for a, b in zip(whole, part):
        assert torch.equal(a, b)
    for a, b in zip(gwhole[:3], gpart[:3]):
        assert torch.equal(a, b)
    # Two orders of one sum: each within 160u of sum |z x r| (see above), whose terms have a mean below 4.
    for a, b, n in zip(gwhole[3:], gpart[3:], (hq, hkv)):
        assert float((a - b).abs().max()) <= 320 * U * sum(docs) * n * 4


def test_a_shard_without_tokens(cuda):
    """Its weight gradients are zeros where they are written, and nothing else is."""
    from context_document_masked_gb300 import fcp
    docs, hq, hkv, d = [1], 2, 1, 64
    qkv, w, f, (dq, dk, _) = make(docs, hq, hkv, d, d, seed=2)
    s = session(docs, 2, hq, hkv, d)
    empty = [j for j in range(2) if s.plan.shard(j)["tokens"] == 0][0]
    x = qkv.cuda()
    out = [torch.full((1, h, d), 3.0, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv)]
    gw = [torch.full((d,), 3.0, device="cuda") for _ in range(2)]
    args = (dq.cuda(), dk.cuda(), None, *slices(x, hq, hkv)[:2], s.dplan, empty, *out, None, *gw, s.ws)
    kw = dict(wq=w[0].cuda(), wk=w[1].cuda(), inv_freq=f.cuda())
    fcp.qk_norm_rope_bwd(*args, **kw, add_dw=True)
    assert all((t == 3).all() for t in out + gw)
    fcp.qk_norm_rope_bwd(*args, **kw)
    assert all((t == 3).all() for t in out) and all((t == 0).all() for t in gw)
    s.qk_norm_rope(*slices(x, hq, hkv)[:2], **kw, shard=empty, q=out[0], k=out[1])
    assert all((t == 3).all() for t in out)


def test_in_place_and_equal_bits_twice(cuda):
    docs, hq, hkv, d = [500, 12], 4, 2, 128
    qkv, w, f, (dq, dk, dv) = make(docs, hq, hkv, d, d, seed=9)
    s = session(docs, 2, hq, hkv, d)
    x = qkv.cuda()
    kw = dict(wq=w[0].cuda(), wk=w[1].cuda(), inv_freq=f.cuda())
    g = [t.cuda() for t in (dq, dk, dv)]
    a = s.qk_norm_rope(*slices(x, hq, hkv), **kw)
    own = [t.contiguous() for t in slices(x, hq, hkv)]
    s.qk_norm_rope(*own, **kw, q=own[0], k=own[1], v=own[2])
    for m, n in zip(a, own):
        assert torch.equal(m, n)
    first = s.qk_norm_rope_backward(*g, *slices(x, hq, hkv)[:2], **kw)
    added = torch.full_like(first[3], 2.0)
    both = s.qk_norm_rope_backward(*g, *slices(x, hq, hkv)[:2], **kw, dwq=added)
    assert both[3] is added and torch.equal(added, first[3] + 2.0) and torch.equal(both[4], first[4])
    again = s.qk_norm_rope_backward(*g, *slices(x, hq, hkv)[:2], **kw)
    for m, n in zip(first, again):
        assert torch.equal(m, n)
    parts = slices(x, hq, hkv)       # the gradient over the projection itself
    s.qk_norm_rope_backward(*g, parts[0], parts[1], **kw, dq_in=parts[0], dk_in=parts[1], dv_in=parts[2])
    for m, n in zip(first, parts):
        assert torch.equal(m, n)


def test_captured_replayed_and_on_another_stream(cuda):
    docs, hq, hkv, d = [700, 1, 323], 8, 2, 64
    qkv, w, f, (dq, dk, dv) = make(docs, hq, hkv, d, 32, seed=10)
    s = session(docs, 2, hq, hkv, d)
    x, other = qkv.cuda(), qkv.flip(0).contiguous().cuda()
    kw = dict(wq=w[0].cuda(), wk=w[1].cuda(), inv_freq=f.cuda(), interleaved=True)
    g = [t.cuda() for t in (dq, dk, dv)]

    def step(src):
        return (*s.qk_norm_rope(*slices(src, hq, hkv), **kw),
                *s.qk_norm_rope_backward(*g, *slices(src, hq, hkv)[:2], **kw))
    want = [[t.clone() for t in step(y)] for y in (x, other)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a, b in zip(step(x), want[0]):
            assert torch.equal(a, b)
    torch.cuda.current_stream().wait_stream(side)
    src = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(src)
    for y, ref in ((other, want[1]), (x, want[0]), (other, want[1])):
        src.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a, b)


def test_infinities_and_zeros_stay_in_their_head(cuda):
    """An infinite or all-zero head gives NaN or zeros there, as the formula
    does, and touches no other head or token."""
    docs, hq, hkv, d = [70], 6, 2, 128
    qkv, w, f, _ = make(docs, hq, hkv, d, d, seed=11)
    s = session(docs, 1, hq, hkv, d)
    kw = dict(wq=w[0].cuda(), wk=w[1].cuda(), inv_freq=f.cuda())
    clean = s.qk_norm_rope(*slices(qkv.cuda(), hq, hkv), **kw)
    bad = qkv.clone()
    bad[3, 2] = 0
    bad[9, 4, 7] = float("inf")
    bad[11, 7, 0] = float("nan")
    got = s.qk_norm_rope(*slices(bad.cuda(), hq, hkv), **kw)
    assert (got[0][3, 2] == 0).all()
    assert torch.isnan(got[0][9, 4]).any() and torch.isnan(got[1][11, 1]).all()
    for i, touched in ((0, [(3, 2), (9, 4)]), (1, [(11, 1)])):
        m = torch.ones_like(got[i], dtype=torch.bool)
        for t, h in touched:
            m[t, h] = False
        assert torch.equal(got[i][m], clean[i][m])


def test_wide_strides_pass_32_bits(cuda):
    """Rows 40,000 elements apart over 60,000 tokens: the last offsets are past
    2^31 elements."""
    T, hq, hkv, d, stride = 60_000, 2, 1, 64, 40_000
    big = torch.empty(T, stride, dtype=torch.bfloat16, device="cuda")
    heads = torch.as_strided(big, (T, 4, d), (stride, d, 1))
    small = torch.randn(T, 4, d, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(torch.bfloat16)
    heads.copy_(small)
    s = session([T], 1, hq, hkv, d)
    f = torch.tensor([0.5] * 32, device="cuda")
    a = s.qk_norm_rope(*slices(heads, hq, hkv), inv_freq=f)
    b = s.qk_norm_rope(*slices(small, hq, hkv), inv_freq=f)
    for m, n in zip(a, b):
        assert torch.equal(m, n)


def test_refusals_on_gpu_tensors(cuda):
    docs, hq, hkv, d = [64], 4, 2, 64
    qkv, w, f, (dq, dk, dv) = make(docs, hq, hkv, d, d, seed=12)
    s = session(docs, 1, hq, hkv, d)
    x = qkv.cuda()
    q, k, v = slices(x, hq, hkv)
    for bad in (dict(q_in=q.float()), dict(q_in=q.transpose(1, 2)), dict(k_in=k[:63]), dict(k_in=x[:, hq:hq + 1]),
                dict(v_in=v, v=v.contiguous().float()), dict(wq=w[0].cuda(), wk=w[1].cuda().to(torch.bfloat16)),
                dict(wq=w[0][:32].cuda()), dict(inv_freq=f.cuda().double()), dict(inv_freq=f),
                dict(q_in=torch.as_strided(x, (64, hq, d), (hq * d - 8, d, 1)))):
        with pytest.raises(ValueError):
            s.qk_norm_rope(**{"q_in": q, "k_in": k, **bad})
    from context_document_masked_gb300 import fcp
    with pytest.raises(fcp.FcpError):
        s.qk_norm_rope(q, k, inv_freq=torch.ones(12, device="cuda"))          # rot_dim 24
    with pytest.raises(fcp.FcpError):
        s.qk_norm_rope(q, k, wq=w[0].cuda(), norm=False)
    with pytest.raises(ValueError):
        s.qk_norm_rope_backward(dq.cuda(), dk.cuda().to(torch.bfloat16), None, q, k)
    with pytest.raises(ValueError):
        s.qk_norm_rope_backward(dq.cuda(), dk.cuda(), None, q, k, dv_in=v)
