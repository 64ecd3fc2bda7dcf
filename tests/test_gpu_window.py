"""Attention under a sliding window with sinks on the GPU, and its gradients,
against the definition in 64 bits.

Bounds, element by element (u = 2^-24, fp32's half step; h = 2^-11, fp16's;
bf16's is 2^-8), for the arithmetic that the kernels are documented to do, n the
keys that a row sees at most (in dV and dK the queries that see a key):
  scores    d products summed in fp32 and four more steps, on |q| |k| scale:
            e_s = (d + 8) 2u max(|q| |k|) scale + 2^-21 (the exponential), a
            relative error of every probability;
  LSE       e_s + (n + 8) 2u;
  O         P in fp16 beside V: (h + 2 e_s + n 2u) P|V| + n 2^-25 max|V|;
  dV        the same with P^T |dO|;
  dS        P, dP - D and their product in fp16: (3h + 2 e_s) |dS|, and P times
            the error of dP - D, which is (d + 2) 2u |dO||V| + |dO| err(O);
            values below fp16's normal range add 2^-24 (1 + |dP - D|);
  dQ, dK    scale (err(dS) + n 2u |dS|) times |K|, |Q|."""
import math

import numpy as np
import pytest
import torch

import synth
from oracle import attention as A
from oracle import window as W

pytestmark = pytest.mark.gpu

U, H, BF16 = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8


def session(docs, cp, policy, hq, hkv, d, window, sinks, **kw):
    from context_document_masked_gb300.session import CPAttention
    return CPAttention(docs, cp, policy, hq, hkv, d, window=window, sinks=sinks, **kw)


def make(docs, hq, hkv, d, seed):
    T = sum(docs)
    return (*synth.make_qkv(T, hq, hkv, d, seed=seed), synth.make_dout(T, hq, d, seed=seed))


def reference(q, k, v, do, docs, window, sinks, scale=None, kv_block=None):
    """Results and bounds, document by document and head by head."""
    q, k, v, do = (A.to_f64(x) for x in (q, k, v, do))
    T, hq, d = q.shape
    G, scale = hq // k.shape[1], scale or 1 / math.sqrt(d)
    lo, hi = kv_block or (0, T)
    zero = lambda *s: (np.zeros(s), np.zeros(s))  # noqa: E731
    o, lse, dq = zero(T, hq, d), zero(hq, T), zero(T, hq, d)
    dk, dv = zero(*k.shape), zero(*v.shape)
    a = 0
    for n in docs:
        e = a + n
        key = np.arange(a, e)
        seen = W.visible(n, window, sinks) & (key >= lo) & (key < hi)
        rows, cols = seen.sum(1).max(), seen.sum(0).max()
        for h in range(hq):
            Q, K, V, dO = q[a:e, h], k[a:e, h // G], v[a:e, h // G], do[a:e, h]
            s = np.where(seen, scale * Q @ K.T, -np.inf)
            m = s.max(1)
            some = np.isfinite(m)
            m = np.where(some, m, 0)
            p = np.exp(s - m[:, None])
            l = np.where(some, p.sum(1), 1)
            p /= l[:, None]
            es = (d + 8) * 2 * U * scale * (np.abs(Q) @ np.abs(K).T).max() + 2.0 ** -21
            O = p @ V
            eO = (H + 2 * es + rows * 2 * U) * (p @ np.abs(V)) + rows * 2.0 ** -25 * np.abs(V).max()
            o[0][a:e, h], o[1][a:e, h] = O, eO
            lse[0][h, a:e], lse[1][h, a:e] = np.where(some, m + np.log(l), -np.inf), es + (rows + 8) * 2 * U
            x = dO @ V.T - (dO * O).sum(1, keepdims=True)
            ds = p * x
            ex = (d + 2) * 2 * U * (np.abs(dO) @ np.abs(V).T) + (np.abs(dO) * eO).sum(1, keepdims=True)
            eds = (3 * H + 2 * es) * np.abs(ds) + p * ex + 2.0 ** -24 * (1 + np.abs(x)) * (p > 0)
            eds = eds + max(rows, cols) * 2 * U * np.abs(ds)
            dq[0][a:e, h], dq[1][a:e, h] = scale * ds @ K, scale * eds @ np.abs(K)
            dk[0][a:e, h // G] += scale * ds.T @ Q
            dk[1][a:e, h // G] += scale * eds.T @ np.abs(Q)
            dv[0][a:e, h // G] += p.T @ dO
            dv[1][a:e, h // G] += (H + 2 * es + cols * 2 * U) * (p.T @ np.abs(dO)) + cols * 2.0 ** -24 * np.abs(dO).max()
        a = e
    return dict(out=o, lse=lse, dq=dq, dk=dk, dv=dv)


def within(got, want, name, extra=0.0):
    ref, err = want[name]
    g = A.to_f64(got)
    inf = ~np.isfinite(ref)
    assert np.array_equal(g[inf], ref[inf]), name
    g, ref = np.where(inf, 0, g), np.where(inf, 0, ref)
    over = np.abs(g - ref) - err - extra * np.abs(ref)
    assert (over <= 1e-30).all(), f"{name}: {float(over.max())} over its bound"


def step(s, x):
    q, k, v, do = x
    s.gather(k, v)
    out, lse = s.forward(q, k, v, out_dtype=torch.float32)
    return out, lse, *s.backward(q, k, v, out, lse, do)


NAMES = ("out", "lse", "dq", "dk", "dv")
CASES = [
    # documents, cp, policy, hq, hkv, d, window, sinks
    (synth.doc_lengths(1), 2, "llama3", 4, 2, 64, 128, 4),
    (synth.doc_lengths(1), 2, "hybrid", 4, 2, 128, 100, 0),
    ([1, 127, 128, 129, 255, 256, 1, 1, 600, 2], 3, "perdoc", 4, 2, 128, 64, 4),
    ([1, 127, 128, 129, 255, 256, 1, 1, 600, 2], 2, "perdoc", 6, 2, 64, 1, 0),
    ([1, 127, 128, 129, 255, 256, 1, 1, 600, 2], 1, "perdoc", 4, 1, 128, 1, 1),
    ([1200], 4, "perdoc", 5, 5, 64, 128, 8),
    ([1200], 8, "perdoc", 4, 2, 128, 300, 64),
    ([1201], 1, "perdoc", 2, 2, 128, 5000, 4),
    ([700, 500], 2, "wholedoc", 8, 1, 64, 129, 16),
    ([9, 20, 31, 40], 4, "perdoc", 4, 2, 64, 3, 7),
    ([40, 24], 8, "llama3", 4, 4, 128, 2, 20),
    ([64] * 9 + [37], 3, "perdoc", 3, 1, 128, 31, 33),
    ([2500, 3], 2, "perdoc", 4, 2, 64, 700, 1),
    ([300] * 4, 2, "hybrid", 2, 1, 64, 2 ** 31 - 1, 3),
    ([1], 1, "perdoc", 4, 2, 64, 1, 4),
]


@pytest.mark.parametrize("docs,cp,policy,hq,hkv,d,window,sinks", CASES)
def test_forward_and_gradients(cuda, docs, cp, policy, hq, hkv, d, window, sinks):
    x = make(docs, hq, hkv, d, seed=len(docs) + d)
    want = reference(*x, docs, window, sinks)
    s = session(docs, cp, policy, hq, hkv, d, window, sinks)
    xd = [t.cuda() for t in x]
    got = step(s, xd)
    assert s.device_status() == 0
    for name, y in zip(NAMES, got):
        within(y.cpu(), want, name)
    out16, lse16 = s.forward(*xd[:3])
    within(out16.cpu(), want, "out", extra=BF16)
    assert torch.equal(lse16, got[1])


@pytest.mark.parametrize("docs,cp,policy,hq,hkv,d,window,sinks", [CASES[0], CASES[2], CASES[6], CASES[9], CASES[11]])
def test_one_shard_at_a_time(cuda, docs, cp, policy, hq, hkv, d, window, sinks):
    """Shard by shard, with workspaces and buffers that hold NaN where nothing is promised: outputs only at the shard's
    rows, dK and dV added up."""
    x = make(docs, hq, hkv, d, seed=7)
    want = reference(*x, docs, window, sinks)
    s = session(docs, cp, policy, hq, hkv, d, window, sinks)
    q, k, v, do = (t.cuda() for t in x)
    s.ws[64:] = -1  # NaN in every type, behind the header
    T = sum(docs)
    nan = dict(device="cuda", dtype=torch.float32)
    out, lse = torch.full((T, hq, d), math.nan, **nan), torch.full((hq, T), math.nan, **nan)
    dq = torch.full((T, hq, d), math.nan, **nan)
    dk, dv = torch.zeros(T, hkv, d, **nan), torch.zeros(T, hkv, d, **nan)
    done = torch.zeros(T, dtype=torch.bool, device="cuda")
    for j in range(cp):
        rows = torch.from_numpy(s.plan.query_indices(j)).cuda().long()
        if len(rows) == 0:
            continue
        s.kbuf.view(torch.int16).fill_(-1)
        s.vbuf.view(torch.int16).fill_(-1)
        s.gather(k, v, shard=j)
        s.forward(q, k, v, shard=j, out=out, lse=lse)
        done[rows] = True
        assert torch.equal(out.isnan().any(2).any(1), ~done) and torch.equal(lse.isnan().any(0), ~done)
        s.ws[64:] = -1
        before = dq.clone()
        s.backward(q, k, v, out, lse, do, shard=j, dq=dq, dk=dk, dv=dv, zero_kv_grads=False)
        assert torch.equal(dq.isnan().any(2).any(1), ~done)
        other = done.clone()
        other[rows] = False
        assert torch.equal(dq[other], before[other])
    assert s.device_status() == 0
    for name, y in zip(NAMES, (out, lse, dq, dk, dv)):
        within(y.cpu(), want, name)


@pytest.mark.parametrize("window,sinks", [(70, 4), (130, 0), (5, 64)])
def test_key_blocks_merge(cuda, window, sinks):
    """Partial results over key blocks, rows without a key in a block among them."""
    from context_document_masked_gb300 import fcp
    docs, cp, hq, hkv, d = [500, 3, 297], 2, 4, 2, 128
    x = make(docs, hq, hkv, d, seed=3)
    s = session(docs, cp, "perdoc", hq, hkv, d, window, sinks)
    q, k, v, _ = (t.cuda() for t in x)
    s.gather(k, v)
    T = sum(docs)
    parts, lses = [], []
    for block in ((0, 2), (2, 333), (333, 333), (333, 801 - 1)):
        out, lse = s.forward(q, k, v, kv_block=block, out_dtype=torch.float32)
        want = reference(*x, docs, window, sinks, kv_block=block)
        within(out.cpu(), want, "out")
        within(lse.cpu(), want, "lse")
        parts.append(out)
        lses.append(lse)
    merged, lse = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(hq, T, device="cuda")
    fcp.merge(torch.stack(parts), torch.stack(lses), merged, lse)
    want = reference(*x, docs, window, sinks)
    # The merge adds a few roundings of its own weights.
    within(lse.cpu(), {"lse": (want["lse"][0], want["lse"][1] + 16 * U * 8)}, "lse")
    within(merged.cpu(), {"out": (want["out"][0], 2 * want["out"][1] + 2.0 ** -20)}, "out", extra=BF16)


def test_large_scores(cuda):
    """Scores that grow and fall along the document: rescales, rows whose first tiles hold no key of theirs, and masked
    scores far above the row's own."""
    docs, hq, hkv, d, window, sinks = [900, 411], 4, 2, 128, 200, 4
    q, k, v, do = make(docs, hq, hkv, d, seed=11)
    ramp = torch.cat([1 + 1.5 * torch.arange(n) / n if i == 0 else 2.5 - 1.5 * torch.arange(n) / n
                      for i, n in enumerate(docs)])
    q, k = (2 * q.float()).bfloat16(), (k.float() * ramp[:, None, None]).bfloat16()
    want = reference(q, k, v, do, docs, window, sinks)
    s = session(docs, 2, "perdoc", hq, hkv, d, window, sinks)
    for name, y in zip(NAMES, step(s, [t.cuda() for t in (q, k, v, do)])):
        within(y.cpu(), want, name)


def test_closed_form(cuda):
    """Q = 0: every row attends to its keys alike."""
    n, window, sinks, hq, hkv, d = 1000, 150, 5, 2, 1, 64
    _, k, v, do = make([n], hq, hkv, d, seed=2)
    s = session([n], 4, "perdoc", hq, hkv, d, window, sinks)
    q = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    out, lse, _, dk, _ = step(s, [q, *(t.cuda() for t in (k, v, do))])
    seen = torch.from_numpy(W.visible(n, window, sinks)).double()
    count = seen.sum(1)
    mean = (seen @ v[:, 0].double()) / count[:, None]
    # P is a power of two times 1 (exact in fp16), V exact; fp32 sums of at most 155 values below 6.
    assert (out.cpu().double() - mean[:, None]).abs().max() < 160 * 2 * U * 6
    assert (lse.cpu().double() - count.log()).abs().max() < 4e-6
    assert dk.abs().max().item() == 0.0


def test_a_wide_window_is_the_attention(cuda):
    """Bit for bit where the tiles are the same."""
    docs, hq, hkv, d = [700, 1, 333], 4, 2, 128
    x = [t.cuda() for t in make(docs, hq, hkv, d, seed=5)]
    a, b = session(docs, 1, "perdoc", hq, hkv, d, 0, 0), session(docs, 1, "perdoc", hq, hkv, d, 700, 0)
    (o1, l1, *g1), (o2, l2, *g2) = step(a, x), step(b, x)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    for y, z in zip(g1, g2):  # added up by atomics, in any order
        torch.testing.assert_close(y, z, atol=2e-5, rtol=2e-5)


def test_sessions_of_one_sequence_share_shards_and_workspace(cuda):
    """Layers with different windows in turn, one workspace, and a new plan for the next sequence."""
    docs, cp, hq, hkv, d = [900, 124, 1000], 4, 4, 2, 64
    x = make(docs, hq, hkv, d, seed=9)
    xd = [t.cuda() for t in x]
    layers = [session(docs, cp, "hybrid", hq, hkv, d, w, s) for w, s in ((0, 0), (64, 4), (500, 0))]
    ws = max((a.ws for a in layers), key=lambda w: w.numel())
    for a in layers:
        a.ws = ws
        assert all(a.plan.shard(j)["pieces"] == layers[0].plan.shard(j)["pieces"] for j in range(cp))
    for a in layers * 2:
        want = reference(*x, docs, a.window or 10 ** 6, a.sinks)
        for name, y in zip(NAMES, step(a, xd)):
            within(y.cpu(), want, name)
    docs = [24, 1500, 500]
    a = layers[1]
    a.set_plan(docs)
    assert a.plan.window == 64 and a.plan.sinks == 4
    want = reference(*x, docs, 64, 4)
    for name, y in zip(NAMES, step(a, xd)):
        within(y.cpu(), want, name)


def test_captured_steps_on_another_stream(cuda):
    """A graph of gather, forward and backward replayed with new inputs beside eager calls on the current stream."""
    docs, cp, hq, hkv, d, window, sinks = [800, 224], 2, 4, 2, 128, 96, 4
    a, b = (session(docs, cp, "perdoc", hq, hkv, d, window, sinks) for _ in range(2))
    x1, x2 = (make(docs, hq, hkv, d, seed=i) for i in (1, 2))
    bufs = [t.cuda() for t in x1]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(a, bufs)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        captured = step(a, bufs)
    for t, y in zip(bufs, x2):
        t.copy_(y)
    graph.replay()
    eager = step(b, [t.cuda() for t in x1])
    torch.cuda.synchronize()
    for got, x in ((captured, x2), (eager, x1)):
        want = reference(*x, docs, window, sinks)
        for name, y in zip(NAMES, got):
            within(y.cpu(), want, name)


def test_refusals(cuda):
    from context_document_masked_gb300 import fcp
    docs, hq, hkv, d = [100, 28], 4, 2, 128
    q, k, v, _ = (t.cuda() for t in make(docs, hq, hkv, d, seed=1))
    s = session(docs, 1, "perdoc", hq, hkv, d, 32, 4)
    for call in (lambda: s.forward_ring(q, k, v), lambda: s.forward_qk8(q, k, v),
                 lambda: s.forward_bias(q, k, v, torch.zeros(hq, 1, device="cuda"), [0])):
        with pytest.raises(fcp.FcpError) as e:
            call()
        assert e.value.status == fcp.ERR_UNSUPPORTED


def test_wait_that_gives_up(cuda):
    """A bounded wait that expires is reported, and the next call is right."""
    from context_document_masked_gb300 import fcp
    docs, hq, hkv, d, window, sinks = [400], 4, 2, 64, 64, 4
    x = make(docs, hq, hkv, d, seed=4)
    xd = [t.cuda() for t in x]
    s = session(docs, 1, "perdoc", hq, hkv, d, window, sinks)
    fcp.debug_set_wait_limit(-1)
    try:
        s.forward(*xd[:3])
        assert s.device_status() == fcp.ERR_TIMEOUT
    finally:
        fcp.debug_set_wait_limit(0)
    want = reference(*x, docs, window, sinks)
    for name, y in zip(NAMES, step(s, xd)):
        within(y.cpu(), want, name)
