"""Attention with a bucketed distance bias on the GPU, and its gradients,
against the definition in 64 bits.

Bounds, element by element (u = 2^-24, fp32's half step; h = 2^-11, fp16's;
bf16's is 2^-8), for the arithmetic that the kernels are documented to do:
  scores    d products summed in fp32 and four more steps, on |q| |k| scale and
            on |b|: e_s = (d + 8) 2u max(|q| |k|) scale + 8u max|b| + 2^-21 (the
            exponential), a relative error of every probability;
  LSE       e_s + (n + 8) 2u;
  O         P in fp16 beside V: (h + 2 e_s + n 2u) P|V| + n 2^-25 max|V|;
  dV        the same with P^T |dO|;
  dS        P, dP - D and their product in fp16: (3h + 2 e_s) |dS|, and P times
            the error of dP - D, which is (d + 2) 2u |dO||V| + |dO| err(O);
            values below fp16's normal range add 2^-24 (1 + |dP - D|);
  dQ, dK    scale (err(dS) + n 2u |dS|) times |K|, |Q|;
  dbias     err(dS) + n 2u |dS|, summed over the bucket's pairs."""
import math

import numpy as np
import pytest
import torch

import synth
from oracle import attention as A
from oracle import positions as N

pytestmark = pytest.mark.gpu

U, H, BF16 = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8
LOW = float(np.finfo(np.float32).min)


def session(docs, cp, hq, hkv, d, policy="perdoc"):
    from context_document_masked_gb300.session import CPAttention
    return CPAttention(docs, cp, policy, hq, hkv, d)


def make(docs, hq, hkv, d, n, seed, spread=1.0):
    T = sum(docs)
    q, k, v = synth.make_qkv(T, hq, hkv, d, seed=seed)
    do = synth.make_dout(T, hq, d, seed=seed)
    b = torch.randn(hq, n, generator=torch.Generator().manual_seed(seed)) * spread
    return q, k, v, do, b


def reference(q, k, v, do, b, starts, docs, scale=None):
    """Results and bounds, document by document and head by head."""
    q, k, v, do, b = (A.to_f64(x) for x in (q, k, v, do, b))
    b = np.where(b <= -1e6, -np.inf, b)
    T, hq, d = q.shape
    G, scale = hq // k.shape[1], scale or 1 / math.sqrt(d)
    zero = lambda *s: (np.zeros(s), np.zeros(s))  # noqa: E731
    o, lse, dq, db = zero(T, hq, d), zero(hq, T), zero(T, hq, d), zero(*b.shape)
    dk, dv = zero(*k.shape), zero(*v.shape)
    big_b = np.abs(b[np.isfinite(b)]).max(initial=0)
    a = 0
    for n in docs:
        e = a + n
        dist = np.arange(n)[:, None] - np.arange(n)
        bucket = N.bucket_of(np.maximum(dist, 0), starts)
        for h in range(hq):
            Q, K, V, dO = q[a:e, h], k[a:e, h // G], v[a:e, h // G], do[a:e, h]
            s = np.where(dist >= 0, scale * Q @ K.T + b[h][bucket], -np.inf)
            m = s.max(1)
            seen = np.isfinite(m)
            m = np.where(seen, m, 0)
            p = np.exp(s - m[:, None])
            l = np.where(seen, p.sum(1), 1)
            p /= l[:, None]
            es = (d + 8) * 2 * U * scale * (np.abs(Q) @ np.abs(K).T).max() + 8 * U * big_b + 2.0 ** -21
            O = p @ V
            eO = (H + 2 * es + n * 2 * U) * (p @ np.abs(V)) + n * 2.0 ** -25 * np.abs(V).max()
            o[0][a:e, h], o[1][a:e, h] = O, eO
            lse[0][h, a:e], lse[1][h, a:e] = np.where(seen, m + np.log(l), -np.inf), es + (n + 8) * 2 * U
            x = dO @ V.T - (dO * O).sum(1, keepdims=True)
            ds = p * x
            ex = (d + 2) * 2 * U * (np.abs(dO) @ np.abs(V).T) + (np.abs(dO) * eO).sum(1, keepdims=True)
            eds = (3 * H + 2 * es) * np.abs(ds) + p * ex + 2.0 ** -24 * (1 + np.abs(x)) * (p > 0)
            eds = eds + n * 2 * U * np.abs(ds)
            dq[0][a:e, h], dq[1][a:e, h] = scale * ds @ K, scale * eds @ np.abs(K)
            dk[0][a:e, h // G] += scale * ds.T @ Q
            dk[1][a:e, h // G] += scale * eds.T @ np.abs(Q)
            dv[0][a:e, h // G] += p.T @ dO
            dv[1][a:e, h // G] += (H + 2 * es + n * 2 * U) * (p.T @ np.abs(dO)) + n * 2.0 ** -24 * np.abs(dO).max()
            np.add.at(db[0][h], bucket[dist >= 0], ds[dist >= 0])
            np.add.at(db[1][h], bucket[dist >= 0], eds[dist >= 0])
        a = e
    return dict(out=o, lse=lse, dq=dq, dk=dk, dv=dv, dbias=db)


def within(got, want, name, extra=0.0):
    ref, err = want[name]
    g = A.to_f64(got)
    inf = ~np.isfinite(ref)
    assert np.array_equal(g[inf], ref[inf]), name
    g, ref = np.where(inf, 0, g), np.where(inf, 0, ref)
    over = np.abs(g - ref) - err - extra * np.abs(ref)
    assert (over <= 1e-30).all(), f"{name}: {float(over.max())} over its bound"


def step(s, x, starts, **kw):
    q, k, v, do, b = x
    s.gather(k, v)
    out, lse = s.forward_bias(q, k, v, b, starts, out_dtype=torch.float32)
    return out, lse, *s.backward_bias(q, k, v, out, lse, do, b, starts, **kw)


CASES = [
    # name, documents, cp, policy, hq, hkv, d, bucket starts (a pair: the usual ones), spread of the biases
    ("usual", synth.doc_lengths(1), 2, "llama3", 4, 2, 64, (32, 128), 1.0),
    ("tile_edges", [1, 127, 128, 129, 255, 256, 1, 1, 600, 2], 3, "perdoc", 4, 2, 128, (32, 128), 1.0),
    ("one_bucket", [130, 5], 1, "perdoc", 2, 2, 64, [0], 3.0),
    ("itself_and_rest", [300, 1, 211], 2, "perdoc", 2, 1, 128, [0, 1], 2.0),
    ("empty_buckets", [400, 100], 1, "perdoc", 5, 5, 64, [0, 0, 3, 3, 3, 64, 200, 200, 9999], 1.0),
    ("each_its_own", [200, 57], 2, "perdoc", 3, 1, 64, list(range(128)), 1.0),
    ("far_reaching", [1700, 40, 300], 4, "perdoc", 6, 2, 128, (128, 1500), 1.0),
    ("large_biases", [333, 180], 1, "perdoc", 4, 4, 128, (16, 100), 1e3),
    ("many_documents", [1, 2, 3] * 240, 1, "perdoc", 4, 2, 64, (4, 3), 1.0),
    ("mha_wholedoc", [300, 212, 500, 12], 2, "wholedoc", 4, 4, 64, (32, 128), 1.0),
]


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_forward_and_gradients(cuda, case):
    from context_document_masked_gb300 import fcp
    _, docs, cp, policy, hq, hkv, d, starts, spread = case
    starts = fcp.rel_buckets(*starts) if isinstance(starts, tuple) else starts
    x = make(docs, hq, hkv, d, len(starts), seed=hq + d, spread=spread)
    want = reference(*x, starts, docs)
    s = session(docs, cp, hq, hkv, d, policy)
    xc = [t.cuda() for t in x]
    got = step(s, xc, starts)
    out16, lse16 = s.forward_bias(*xc[:3], xc[4], starts)
    torch.cuda.synchronize()
    assert s.device_status() == 0
    for name, t in zip(("out", "lse", "dq", "dk", "dv", "dbias"), got):
        within(t, want, name)
    within(out16, want, "out", BF16)
    assert torch.equal(lse16, got[1])


def test_one_token(cuda):
    x = make([1], 3, 1, 64, 2, seed=1)
    s = session([1], 1, 3, 1, 64)
    out, lse, dq, dk, dv, db = step(s, [t.cuda() for t in x], [0, 1])
    want = reference(*x, [0, 1], [1])
    for name, t in zip(("out", "lse", "dq", "dk", "dv", "dbias"), (out, lse, dq, dk, dv, db)):
        within(t, want, name)


@pytest.mark.parametrize("what", ["window", "not itself", "nothing"])
def test_masked_buckets(cuda, what):
    """-inf, the lowest value and -1e9 mask a bucket: a sliding window, rows that may
    not see themselves (the first of a document sees nothing), nothing at all."""
    docs, hq, hkv, d, starts = [500, 1, 11], 4, 2, 128, [0, 1, 64, 300]
    q, k, v, do, b = make(docs, hq, hkv, d, 4, seed=2)
    if what == "window":
        b[:2, 2:], b[2:, 3] = -math.inf, LOW
    elif what == "not itself":
        b[::2, 0], b[1::2, 0] = -1e9, LOW
    else:
        b[1], b[3] = -math.inf, LOW
    want = reference(q, k, v, do, b, starts, docs)
    s = session(docs, 2, hq, hkv, d)
    got = step(s, [t.cuda() for t in (q, k, v, do, b)], starts)
    assert s.device_status() == 0
    for name, t in zip(("out", "lse", "dq", "dk", "dv", "dbias"), got):
        within(t, want, name)
    if what != "window":
        empty = torch.from_numpy(~np.isfinite(want["lse"][0])).cuda()
        assert empty.any() and (got[0].transpose(0, 1)[empty] == 0).all() and (got[2].transpose(0, 1)[empty] == 0).all()
    masked = (b <= -1e6).cuda()
    assert (got[5][masked] == 0).all()


def test_key_blocks_merge_and_shards(cuda):
    """Partial results over key blocks merge to the whole; shard by shard the
    forward has the same bits, and the gradients add up to within their bounds."""
    from context_document_masked_gb300 import fcp
    docs, cp, hq, hkv, d = [700, 1, 40, 283], 4, 4, 2, 128
    starts = fcp.rel_buckets(32, 128)
    x = make(docs, hq, hkv, d, 32, seed=3)
    want = reference(*x, starts, docs)
    q, k, v, do, b = xc = [t.cuda() for t in x]
    s = session(docs, cp, hq, hkv, d, "perdoc")
    whole = step(s, xc, starts)
    T = sum(docs)
    parts = [s.forward_bias(q, k, v, b, starts, kv_block=blk, out_dtype=torch.float32)
             for blk in ((0, 333), (333, 334), (334, 900), (900, T))]
    out, lse = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(hq, T, device="cuda")
    fcp.merge(torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]), out, lse)
    want["out"] = (want["out"][0], 2 * want["out"][1])      # the block's error and the merge's
    want["lse"] = (want["lse"][0], 2 * want["lse"][1])
    within(out, want, "out", BF16)
    within(lse, want, "lse")
    o, l = torch.full_like(whole[0], 7.0), torch.full_like(whole[1], 7.0)
    g = [torch.full_like(whole[2], 7.0)] + [torch.zeros_like(t) for t in whole[3:]]
    for j in range(cp):
        s.gather(k, v, shard=j)
        s.forward_bias(q, k, v, b, starts, shard=j, out=o, lse=l, out_dtype=torch.float32)
        s.backward_bias(q, k, v, o, l, do, b, starts, shard=j, dq=g[0], dk=g[1], dv=g[2], dbias=g[3], zero_grads=False)
    assert torch.equal(o, whole[0]) and torch.equal(l, whole[1]) and s.device_status() == 0
    for name, t in zip(("dq", "dk", "dv", "dbias"), g):
        within(t, want, name)


@pytest.mark.parametrize("scale", [0.3, 1e-3])
def test_other_scales(cuda, scale):
    """The bias is added after the scale, whatever that is."""
    from context_document_masked_gb300 import fcp
    from context_document_masked_gb300.session import CPAttention
    docs, hq, hkv, d = [333, 1, 178], 4, 2, 64
    starts = fcp.rel_buckets(16, 100)
    x = make(docs, hq, hkv, d, 16, seed=9)
    want = reference(*x, starts, docs, scale=float(np.float32(scale)))
    s = CPAttention(docs, 2, "perdoc", hq, hkv, d, scale=scale)
    for name, t in zip(("out", "lse", "dq", "dk", "dv", "dbias"), step(s, [t.cuda() for t in x], starts)):
        within(t, want, name)


def test_a_shard_without_tokens(cuda):
    """It writes nothing and adds nothing."""
    docs, hq, hkv, d = [1], 2, 1, 64
    q, k, v, do, b = (t.cuda() for t in make(docs, hq, hkv, d, 2, seed=5))
    s = session(docs, 2, hq, hkv, d)
    empty = [j for j in range(2) if s.plan.shard(j)["tokens"] == 0][0]
    full = lambda *n: torch.full(n, 3.0, device="cuda")  # noqa: E731
    out, lse, dq, dk, dv, db = full(1, hq, d), full(hq, 1), full(1, hq, d), full(1, hkv, d), full(1, hkv, d), full(hq, 2)
    s.forward_bias(q, k, v, b, [0, 1], shard=empty, out=out, lse=lse)
    s.backward_bias(q, k, v, out, lse, do, b, [0, 1], shard=empty, dq=dq, dk=dk, dv=dv, dbias=db, zero_grads=False)
    assert all((t == 3).all() for t in (out, lse, dq, dk, dv, db)) and s.device_status() == 0


def test_two_sessions_at_once(cuda):
    """Steps of two sessions on two streams, overlapping."""
    from context_document_masked_gb300 import fcp
    shapes = [([900, 100], 4, 2, 128, (32, 128)), ([700, 3, 321], 6, 3, 64, (16, 200))]
    runs = []
    for n, (docs, hq, hkv, d, bk) in enumerate(shapes):
        starts = fcp.rel_buckets(*bk)
        x = make(docs, hq, hkv, d, len(starts), seed=20 + n)
        runs.append((session(docs, 2, hq, hkv, d), [t.cuda() for t in x], starts, reference(*x, starts, docs), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, xc, starts, _w, st in runs:
            with torch.cuda.stream(st):
                got.append(step(s, xc, starts))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for name, t in zip(("out", "lse", "dq", "dk", "dv", "dbias"), g):
            within(t, runs[i % 2][3], name)


def test_without_a_bias_it_is_the_attention(cuda):
    docs, hq, hkv, d = [900, 124], 8, 2, 128
    x = make(docs, hq, hkv, d, 3, seed=4)
    x[4].zero_()
    want = reference(*x, [0, 40, 500], docs)
    s = session(docs, 2, hq, hkv, d)
    q, k, v, do, b = (t.cuda() for t in x)
    s.gather(k, v)
    out, lse = s.forward(q, k, v, out_dtype=torch.float32)
    within(out, want, "out")
    for name, t in zip(("dq", "dk", "dv"), s.backward(q, k, v, out, lse, do)):
        within(t, want, name)
    for name, t in zip(("out", "lse", "dq", "dk", "dv", "dbias"), step(s, (q, k, v, do, b), [0, 40, 500])):
        within(t, want, name)


def test_captured_with_new_biases_and_on_another_stream(cuda):
    docs, hq, hkv, d, starts = [300, 212], 4, 2, 64, [0, 1, 2, 4, 8, 100]
    x = make(docs, hq, hkv, d, 6, seed=5)
    y = make(docs, hq, hkv, d, 6, seed=6)
    wants = [reference(*z, starts, docs) for z in (x, y)]
    s = session(docs, 2, hq, hkv, d)
    names = ("out", "lse", "dq", "dk", "dv", "dbias")
    xc, yc = [t.cuda() for t in x], [t.cuda() for t in y]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    q, k, v, do, b = yc
    s.gather(k, v, stream=side)
    out, lse = s.forward_bias(q, k, v, b, starts, out_dtype=torch.float32, stream=side)
    got = out, lse, *s.backward_bias(q, k, v, out, lse, do, b, starts, stream=side)
    side.synchronize()
    for name, t in zip(names, got):
        within(t, wants[1], name)
    src = [t.clone() for t in xc]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(s, src, list(starts))
    for z, want in ((yc, wants[1]), (xc, wants[0]), (yc, wants[1])):
        for t, n in zip(src, z):
            t.copy_(n)
        graph.replay()
        for name, t in zip(names, got):
            within(t, want, name)
    assert s.device_status() == 0


@pytest.mark.parametrize("which,hq", [("usual", 2), ("narrow far off", 2), ("usual", 8)])
def test_one_long_document(cuda, which, hq):
    """16,385 tokens on four shards against a plain form in 64 bits on the GPU;
    buckets by logarithms up to 8192, and narrow ones past that."""
    from context_document_masked_gb300 import fcp
    T, hkv, d = 16385, 1, 64
    far = [0, 1, 100, 5000, 8180, 8200, 9000, 9003, 9004, 9040, 9041, 12000, 16300]
    starts = fcp.rel_buckets(64, 8192) if which == "usual" else np.array(far)
    x = make([T], hq, hkv, d, len(starts), seed=7)
    s = session([T], 4, hq, hkv, d)
    xc = [t.cuda() for t in x]
    got = step(s, xc, starts)
    q, k, v, do, b = (t.double() for t in xc)
    dist = torch.arange(T, device="cuda")[:, None] - torch.arange(T, device="cuda")
    bucket = torch.bucketize(dist.clamp(min=0), torch.tensor(starts[1:].tolist(), device="cuda"), right=True)
    dk, dv, edk, edv = torch.zeros_like(k), torch.zeros_like(v), 0, 0
    for h in range(hq):
        p = (q[:, h] @ k[:, 0].T / 8 + b[h][bucket]).masked_fill_(dist < 0, -math.inf)
        lse = torch.logsumexp(p, 1)
        p = p.sub_(lse[:, None]).exp_()
        o = p @ v[:, 0]
        es = (d + 8) * 2 * U * float((q[:, h].abs() @ k[:, 0].abs().T).max()) / 8 + 8 * U * float(b[h].abs().max()) + 2.0 ** -21
        vmax = float(v.abs().max())
        assert float((got[0][:, h] - o).abs().max()) <= (H + 2 * es + T * 2 * U + T * 2.0 ** -25) * vmax
        assert float((got[1][h] - lse).abs().max()) <= es + (T + 8) * 2 * U
        x_ = do[:, h] @ v[:, 0].T - (do[:, h] * o).sum(1, keepdim=True)
        ds = p * x_
        ex = (d + 2) * 2 * U * (do[:, h].abs() @ v[:, 0].abs().T)
        ex += (do[:, h].abs().sum(1, keepdim=True) * (H + 2 * es + T * 2 * U + T * 2.0 ** -25) * vmax)
        eds = (3 * H + 2 * es + T * 2 * U) * ds.abs() + p * ex + 2.0 ** -24 * (1 + x_.abs()) * (p > 0)
        assert ((got[2][:, h] - ds @ k[:, 0] / 8).abs() <= eds @ k[:, 0].abs() / 8).all()
        edk = edk + eds.T @ q[:, h].abs() / 8
        edv = edv + (H + 2 * es + T * 2 * U) * (p.T @ do[:, h].abs()) + T * 2.0 ** -24 * do.abs().max()
        dk[:, 0] += ds.T @ q[:, h] / 8
        dv[:, 0] += p.T @ do[:, h]
        by = torch.zeros(len(starts), dtype=torch.float64, device="cuda").index_add_(0, bucket.flatten(), ds.flatten())
        lim = torch.zeros_like(by).index_add_(0, bucket.flatten(), eds.flatten())
        assert ((got[5][h] - by).abs() <= lim).all()
        del p, x_, ds, eds, ex
    assert ((got[3][:, 0] - dk[:, 0]).abs() <= edk).all() and ((got[4][:, 0] - dv[:, 0]).abs() <= edv).all()


def test_one_workspace_for_other_plans_and_sizes(cuda):
    """A session re-planned (its workspace's regions move) and one workspace used
    for two shapes in turn: nothing that one call leaves reaches the next."""
    from context_document_masked_gb300 import fcp
    hq, hkv, d, starts = 4, 2, 64, [0, 1, 3, 50]
    s = session([500, 12], 2, hq, hkv, d, "hybrid")
    for seed, docs in ((1, [500, 12]), (2, [1] * 100 + [412]), (3, [256, 256]), (4, [512])):
        if seed > 1:
            s.set_plan(docs)
        x = make(docs, hq, hkv, d, 4, seed=seed)
        want = reference(*x, starts, docs)
        for name, t in zip(("out", "lse", "dq", "dk", "dv", "dbias"), step(s, [t.cuda() for t in x], starts)):
            within(t, want, name)
    small, big = ([300, 84], 2, 1, 64), ([700, 68], 6, 3, 128)
    ss = [session(docs, 1, *shape) for docs, *shape in (small, big)]
    ss[0].ws = ss[1].ws
    rows = []
    for k in range(4):
        (docs, *shape), s = (small, big)[k % 2], ss[k % 2]
        x = make(docs, *shape, 4, seed=10 + k)
        want = reference(*x, starts, docs)
        xc = [t.cuda() for t in x]
        for name, t in zip(("out", "lse", "dq", "dk", "dv", "dbias"), step(s, xc, starts)):
            within(t, want, name)
        w = torch.ones(shape[2], device="cuda")
        g = torch.Generator("cuda").manual_seed(5 + k % 2)
        grads = [torch.randn(sum(docs), h, shape[2], device="cuda", generator=g) for h in (shape[0], shape[1])]
        qk = [torch.randn(sum(docs), h, shape[2], device="cuda", generator=g).to(torch.bfloat16) for h in (shape[0], shape[1])]
        rows.append(s.qk_norm_rope_backward(*grads, None, *qk, wq=w, wk=w))
    for a, b in ((0, 2), (1, 3)):
        for m, n in zip(rows[a], rows[b]):
            assert m is None and n is None or torch.equal(m, n)


def test_norm_rope_then_biased_attention(cuda):
    """The path of a layer: projection, head norm (and rotation), attention with
    the bias, and back to the gradients of the projection, the norm weights and
    the bias, against automatic differentiation in 64 bits."""
    from context_document_masked_gb300 import fcp
    docs, cp, hq, hkv, d, rot = [130, 1, 125, 256], 2, 4, 2, 64, 32
    T, n = sum(docs), 16
    starts = fcp.rel_buckets(n, 100)
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    qkv, do = r(T, hq + 2 * hkv, d).to(torch.bfloat16), r(T, hq, d).to(torch.bfloat16)
    wq, wk, b = 1 + 0.1 * r(d), 1 + 0.1 * r(d), r(hq, n)
    f = (1e4 ** (-torch.arange(0, rot, 2) / rot)).float()
    s = session(docs, cp, hq, hkv, d)
    x, dev = qkv.cuda(), [t.cuda() for t in (wq, wk, f, b, do)]
    kw = dict(wq=dev[0], wk=dev[1], inv_freq=dev[2], eps=1e-6)
    q, k, v = s.qk_norm_rope(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], **kw)
    out, lse, dq, dk, dv, db = step(s, (q, k, v, dev[4], dev[3]), starts)
    dx = torch.empty_like(x)
    *_, dwq, dwk = s.qk_norm_rope_backward(dq, dk, dv, x[:, :hq], x[:, hq:hq + hkv], **kw, dq_in=dx[:, :hq],
                                           dk_in=dx[:, hq:hq + hkv], dv_in=dx[:, hq + hkv:])
    assert s.device_status() == 0
    X, W = qkv.double().requires_grad_(), [t.double().requires_grad_() for t in (wq, wk, b)]
    cu = synth.cu_from_lengths(docs)
    pos = torch.from_numpy(N.positions(cu)).double()

    def heads(z, w):
        z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + 1e-6) * w
        c, si = torch.cos(pos[:, None] * f.double())[:, None], torch.sin(pos[:, None] * f.double())[:, None]
        a, e = z[..., :rot // 2], z[..., rot // 2:rot]
        return torch.cat((a * c - e * si, a * si + e * c, z[..., rot:]), -1)
    Q, K, V = heads(X[:, :hq], W[0]), heads(X[:, hq:hq + hkv], W[1]), X[:, hq + hkv:]
    ids = torch.from_numpy(A.doc_ids(cu))
    dist = torch.arange(T)[:, None] - torch.arange(T)
    bucket = torch.bucketize(dist.clamp(min=0), torch.tensor(starts[1:].tolist()), right=True)
    K, V = K.repeat_interleave(2, 1), V.repeat_interleave(2, 1)
    sc = (torch.einsum("ihd,jhd->hij", Q, K) / 8 + W[2][:, bucket]).masked_fill((dist < 0) | (ids[:, None] != ids), -math.inf)
    O = torch.einsum("hij,jhd->ihd", torch.softmax(sc, -1), V)
    ref = torch.autograd.grad((O * do.double()).sum(), [X, *W])
    # Q and K are rounded to bf16 on the way (2^-8 a value, 2^-8 sqrt(2) of a score of size sqrt(d) / 8 = 1):
    # the gradients' norms may be off by a few of these.
    for got, want in ((out, O), (dx, ref[0]), (dwq, ref[1]), (dwk, ref[2]), (db, ref[3])):
        err = (got.cpu().double() - want.detach()).norm() / want.detach().norm()
        assert float(err) <= 4 * BF16


def test_refusals_on_gpu_tensors(cuda):
    docs, hq, hkv, d = [64], 4, 2, 64
    q, k, v, do, b = (t.cuda() for t in make(docs, hq, hkv, d, 2, seed=8))
    s = session(docs, 1, hq, hkv, d)
    from context_document_masked_gb300 import fcp
    for bias, starts in ((b.half(), [0, 1]), (b[:3], [0, 1]), (b, [0, 1, 2]), (b.t().contiguous().t(), [0, 1]), (b.cpu(), [0, 1]),
                         (b, [0.0, 1.0])):
        with pytest.raises(ValueError):
            s.forward_bias(q, k, v, bias, starts)
    for starts in ([1, 2], [0, -1]):
        with pytest.raises((ValueError, fcp.FcpError)):
            s.forward_bias(q, k, v, b, starts)
    out, lse = s.forward_bias(q, k, v, b, [0, 1], out_dtype=torch.float32)
    g = [torch.full_like(t, 5.0) for t in s.backward_bias(q, k, v, out, lse, do, b, [0, 1])]
    given = dict(zip(("dq", "dk", "dv", "dbias"), g))
    want = s.backward_bias(q, k, v, out, lse, do, b, [0, 1])
    for name, t, w in zip(given, s.backward_bias(q, k, v, out, lse, do, b, [0, 1], **given), want):   # set to zero first
        assert t is given[name] and torch.allclose(t, w, rtol=0, atol=1e-5)
    with pytest.raises(ValueError):
        s.backward_bias(q, k, v, out, lse, do, b, [0, 1], dbias=torch.zeros(hq, 3, device="cuda"))
    with pytest.raises(ValueError):
        s.backward_bias(q, k, v, out, lse, do.float(), b, [0, 1])
