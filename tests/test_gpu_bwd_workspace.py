"""The backward in a workspace that other calls have used: it may find anything
behind the header.

A shard's backward loads whole 128-row tiles of the workspace's copies of Q and
dO, rows of other shards among them. Bounds as derived in test_gpu_rel_bias."""
import pytest
import torch

from test_gpu_rel_bias import make, reference, session, within

pytestmark = pytest.mark.gpu

HEADER = 256  # bytes


def shard_by_shard(s, x, starts, biased, before_shard):
    q, k, v, do, b = x
    T, hq, d = q.shape
    out = torch.zeros(T, hq, d, device="cuda")
    lse = torch.zeros(hq, T, device="cuda")
    dq = torch.zeros(T, hq, d, device="cuda")
    dk, dv = (torch.zeros(T, k.shape[1], d, device="cuda") for _ in range(2))
    db = torch.zeros_like(b)
    for j in range(s.cp):
        s.gather(k, v, shard=j)
        before_shard()
        if biased:
            s.forward_bias(q, k, v, b, starts, shard=j, out=out, lse=lse)
        else:
            s.forward(q, k, v, shard=j, out=out, lse=lse)
        before_shard()
        if biased:
            s.backward_bias(q, k, v, out, lse, do, b, starts, shard=j, dq=dq, dk=dk, dv=dv, dbias=db, zero_grads=False)
        else:
            s.backward(q, k, v, out, lse, do, shard=j, dq=dq, dk=dk, dv=dv, zero_kv_grads=False)
    return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv, **(dict(dbias=db) if biased else {}))


CASES = [
    ([700, 1, 40, 283], 4, "perdoc", 4, 2, 64),
    ([130, 5, 300, 77], 4, "wholedoc", 2, 1, 128),      # 512 tokens: pieces of whole documents
    ([1, 2, 3] * 60, 3, "perdoc", 3, 3, 64),            # pieces of a token, many of them inside one tile
    ([129, 127, 128, 256], 5, "llama3", 2, 2, 128),
]


@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
@pytest.mark.parametrize("case", CASES, ids=[c[2] + str(c[4]) + str(len(c[0])) for c in CASES])
def test_nan_behind_the_header(cuda, case, biased):
    docs, cp, policy, hq, hkv, d = case
    starts = [0, 1, 3, 50]
    x = make(docs, hq, hkv, d, 4, seed=31)
    if not biased:
        x[4].zero_()
    want = reference(*x, starts, docs)
    s = session(docs, cp, hq, hkv, d, policy)
    xc = [t.cuda() for t in x]

    def spoil():
        s.ws[HEADER // 4:].fill_(-1)  # NaN in fp32, fp16, bf16 and e4m3
    got = shard_by_shard(s, xc, starts, biased, spoil)
    assert s.device_status() == 0
    for name, t in got.items():
        within(t, want, name)


def test_shapes_in_turn(cuda):
    """One workspace for two shapes, shard by shard: the small one's copies of Q and
    dO lie where the large one left fp32 sums."""
    starts = [0, 1, 3, 50]
    shapes = [([300, 85], 2, 1, 64), ([700, 68], 6, 3, 128)]
    runs = []
    for n, (docs, hq, hkv, d) in enumerate(shapes):
        x = make(docs, hq, hkv, d, 4, seed=40 + n)
        runs.append((session(docs, 3, hq, hkv, d), [t.cuda() for t in x], reference(*x, starts, docs)))
    runs[0][0].ws = runs[1][0].ws
    for k in range(4):
        s, xc, want = runs[1 - k % 2]
        for name, t in shard_by_shard(s, xc, starts, True, lambda: None).items():
            within(t, want, name)
        assert s.device_status() == 0


@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
def test_after_a_wait_that_gave_up(cuda, biased):
    """A backward whose waits give up at once reports it and leaves the header as the
    next call expects it."""
    from context_document_masked_gb300 import fcp
    docs, starts = [300, 1, 83], [0, 1, 3, 50]
    x = make(docs, 4, 2, 64, 4, seed=45)
    if not biased:
        x[4].zero_()
    want = reference(*x, starts, docs)
    s = session(docs, 2, 4, 2, 64)
    q, k, v, do, b = (t.cuda() for t in x)
    s.gather(k, v)
    if biased:
        out, lse = s.forward_bias(q, k, v, b, starts, out_dtype=torch.float32)
        back = lambda d: s.backward_bias(q, k, v, out, lse, d, b, starts)  # noqa: E731
    else:
        out, lse = s.forward(q, k, v, out_dtype=torch.float32)
        back = lambda d: s.backward(q, k, v, out, lse, d)  # noqa: E731
    torch.cuda.synchronize()
    fcp.debug_set_wait_limit(-1)
    try:
        back(do * 1024)
        torch.cuda.synchronize()
        assert s.device_status() == fcp.ERR_TIMEOUT
    finally:
        fcp.debug_set_wait_limit(0)
    assert (s.ws[36:39] == 0).all()  # bytes 144 to 155: the range of the operands
    for name, t in zip(("dq", "dk", "dv", "dbias"), back(do)):
        within(t, want, name)
    assert s.device_status() == 0
