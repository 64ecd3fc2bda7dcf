"""Session calls on a stream that is not the current one: what torch does for a
call (new tensors, zero fills) runs in the order of that stream.

The current stream is kept busy meanwhile, so that work left on it would come
after the call's own. Bounds as derived in test_gpu_rel_bias."""
import pytest
import torch

from test_gpu_rel_bias import make, reference, session, within

pytestmark = pytest.mark.gpu

DOCS, SHAPE = [700, 1, 323], (4, 2, 128)
BUSY = 100_000_000  # cycles of the current stream


@pytest.fixture(scope="module")
def data():
    x = make(DOCS, *SHAPE, 1, seed=21)
    x[4].zero_()
    want = reference(*x, [0], DOCS)
    torch.cuda.synchronize()
    return [t.cuda() for t in x[:4]], want


@pytest.mark.parametrize("given", [False, True], ids=["new", "given"])
def test_step(cuda, data, given):
    (q, k, v, do), want = data
    s = session(DOCS, 2, *SHAPE)
    full = lambda t, *n: torch.full((*t.shape, *n), 5.0, device="cuda")  # noqa: E731
    kw = dict(dq=full(q), dk=full(k), dv=full(v)) if given else {}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    s.gather(k, v, stream=side)
    out, lse = s.forward(q, k, v, out_dtype=torch.float32, stream=side)
    grads = s.backward(q, k, v, out, lse, do, stream=side, **kw)
    with torch.cuda.stream(side):
        got = [t.clone() for t in (out, lse, *grads)]
    torch.cuda.synchronize()
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), got):
        within(t, want, name)
    for name, t in zip(("dq", "dk", "dv"), grads):  # nothing came after the call either
        within(t, want, name)


@pytest.mark.parametrize("how", ["forward", "forward_ring", "forward_qk8"])
def test_outputs_are_made_in_the_streams_order(cuda, data, how):
    """A block that the current stream's queued work has just given back is not the
    other stream's output."""
    (q, k, v, _), want = data
    s = session(DOCS, 2, *SHAPE)
    side = torch.cuda.Stream()
    s.gather(k, v)
    plain = getattr(s, how)(q, k, v, out_dtype=torch.float32)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    old = [torch.full_like(t, 7.0) for t in plain]  # written when the sleep ends
    del old
    got = getattr(s, how)(q, k, v, out_dtype=torch.float32, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(plain, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("which", ["default", "side"])
def test_streams_as_raw_handles(cuda, data, which):
    (q, k, v, do), want = data
    s = session(DOCS, 2, *SHAPE)
    st = torch.cuda.default_stream() if which == "default" else torch.cuda.Stream()
    torch.cuda.synchronize()
    s.gather(k, v, stream=st.cuda_stream)
    out, lse = s.forward(q, k, v, out_dtype=torch.float32, stream=st.cuda_stream)
    got = out, lse, *s.backward(q, k, v, out, lse, do, stream=st.cuda_stream)
    st.synchronize()
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), got):
        within(t, want, name)


def test_set_plan_makes_its_buffers_in_the_streams_order(cuda):
    """A larger workspace starts from zeros on the stream of the plan's upload."""
    docs = [1024]
    x = make(docs, *SHAPE, 1, seed=22)
    x[4].zero_()
    want = reference(*x, [0], docs)
    q, k, v, do = (t.cuda() for t in x[:4])
    s = session([256] * 4, 4, *SHAPE, "wholedoc")
    small = s.ws, s.kbuf
    side = torch.cuda.Stream()
    # Memory whose last writer waits behind the sleep.
    old = [torch.empty(1 << 24, dtype=torch.int32, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for t in old:
        t.fill_(-1)
    del old, t
    s.set_plan(docs, stream=side)
    assert s.ws is not small[0] and s.kbuf is not small[1]
    s.gather(k, v, stream=side)
    out, lse = s.forward(q, k, v, out_dtype=torch.float32, stream=side)
    got = out, lse, *s.backward(q, k, v, out, lse, do, stream=side)
    torch.cuda.synchronize()
    assert s.device_status() == 0
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), got):
        within(t, want, name)
