"""The backward at upstream gradients and values of other sizes.

The gradients are linear in dO (and dQ, dK, dbias in V), and a power of two
changes no significand: what holds for dO holds for 2^e dO, with every bound of
test_gpu_rel_bias times the same power. A loss averaged over a long sequence
gives dO of 2^-17 to 2^-30, where unscaled fp16 operands keep a few bits or
none; large ones would pass fp16's range in dP - D."""
import pytest
import torch

from test_gpu_rel_bias import make, reference, session, within

pytestmark = pytest.mark.gpu

DOCS, STARTS = [333, 1, 178, 512], [0, 1, 2, 9, 100]
NAMES = ("out", "lse", "dq", "dk", "dv", "dbias")


def scaled(want, e_do, e_v):
    """Results and bounds for dO 2^e_do and V 2^e_v."""
    by = dict(out=e_v, lse=0, dq=e_do + e_v, dk=e_do + e_v, dv=e_do, dbias=e_do + e_v)
    return {n: tuple(t * 2.0 ** by[n] for t in pair) for n, pair in want.items()}


def run(s, x, starts, biased):
    q, k, v, do, b = (t.cuda() for t in x)
    s.gather(k, v)
    if biased:
        out, lse = s.forward_bias(q, k, v, b, starts, out_dtype=torch.float32)
        return out, lse, *s.backward_bias(q, k, v, out, lse, do, b, starts)
    out, lse = s.forward(q, k, v, out_dtype=torch.float32)
    return out, lse, *s.backward(q, k, v, out, lse, do)


@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e_do,e_v", [(-20, 0), (-40, 0), (-100, 0), (10, 6), (14, 0), (0, -20), (-20, 12)])
def test_powers_of_two(cuda, e_do, e_v, d, biased):
    q, k, v, do, b = x = make(DOCS, 4, 2, d, len(STARTS), seed=50 + d)
    if not biased:
        b.zero_()
    want = scaled(reference(*x, STARTS, DOCS), e_do, e_v)
    s = session(DOCS, 2, 4, 2, d)
    got = run(s, (q, k, v * 2.0 ** e_v, do * 2.0 ** e_do, b), STARTS, biased)
    if float(do.abs().max()) * 2.0 ** e_do > 65504:  # refused: beyond the fp16 range
        from context_document_masked_gb300 import fcp
        assert s.device_status() == fcp.ERR_UNSUPPORTED
        return
    assert s.device_status() == 0
    if e_v < -10:
        # V's fp16 copies are multiples of 2^-24: off by c = 2^-25 an element, which O keeps (its weights add up to 1),
        # dP and D take times |dO_i|_1 each, and so dS by at most P e, e = 2 c max_i |dO_i|_1. Over the sums of P: 1 a
        # query row, n a key and query head (two a KV head), T over all pairs.
        c, one = 2.0 ** -25, float(do.float().abs().sum(-1).max()) * 2.0 ** e_do
        e, T, n = 2 * c * one, sum(DOCS), max(DOCS)
        more = dict(out=c, lse=0, dv=0, dbias=e * T, dq=e * float(k.abs().max()) / d ** 0.5,
                    dk=e * 2 * n * float(q.abs().max()) / d ** 0.5)
        want = {name: (r, err + more[name]) for name, (r, err) in want.items()}
    for name, t in zip(NAMES, got):
        within(t, want, name)


@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
def test_one_sequence_of_many_sizes(cuda, biased):
    """Gradients of 2^-30 to 1 side by side, zero rows among them: every row of dQ
    within its bound at the largest gradient's size, and no row lost that is
    within 2^-10 of it."""
    docs, d = [512], 64
    q, k, v, do, b = make(docs, 2, 1, d, len(STARTS), seed=60)
    if not biased:
        b.zero_()
    e = (torch.arange(512) % 31).float()
    do = do * (2.0 ** -e)[:, None, None]
    do[5::17] = 0
    do = do.to(torch.bfloat16)
    want = reference(q, k, v, do, b, STARTS, docs)
    s = session(docs, 1, 2, 1, d)
    got = run(s, (q, k, v, do, b), STARTS, biased)
    assert s.device_status() == 0
    for name, t in zip(NAMES, got):
        within(t, want, name)
    dq, ref = got[2].double().cpu(), torch.from_numpy(want["dq"][0])
    near = ((e <= 10) & (do != 0).any(-1).any(-1))[:, None]
    # A row's gradient is a sum of terms each off by 3 2^-11 and more (as above): a twentieth is far outside of that.
    # (The first row sees itself alone: its gradient is zero.)
    good = (dq - ref).norm(dim=-1) <= 0.05 * ref.norm(dim=-1) + 1e-30
    assert (good | ~near)[1:].all()


@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
def test_nothing_comes_back(cuda, biased):
    """dO = 0 gives zeros, and leaves no trace for the next call."""
    x = make(DOCS, 4, 2, 64, len(STARTS), seed=70)
    if not biased:
        x[4].zero_()
    want = reference(*x, STARTS, DOCS)
    s = session(DOCS, 2, 4, 2, 64)
    big = run(s, (*x[:3], x[3] * 2.0 ** 12, x[4]), STARTS, biased)
    zero = run(s, (*x[:3], x[3] * 0, x[4]), STARTS, biased)
    assert all((t == 0).all() for t in zero[2:])
    for name, t in zip(NAMES, run(s, x, STARTS, biased)):
        within(t, want, name)
    for name, t in zip(NAMES, big):
        within(t, scaled(want, 12, 0), name)
    assert s.device_status() == 0


@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
@pytest.mark.parametrize("where", ["do nan", "do inf", "v nan", "v inf"])
def test_one_document_that_is_not_finite(cuda, where, biased):
    """It does not cost the others their bits. Documents of whole tiles on one shard:
    what shares a tile with it has to be finite (P = 0 times NaN is NaN)."""
    docs, d = [256, 128, 384, 256], 64
    q, k, v, do, b = x = make(docs, 4, 2, d, len(STARTS), seed=80)
    if not biased:
        b.zero_()
    want = reference(*x, STARTS, docs)
    name, value = where.split()
    v, do = v.clone(), do.clone()
    {"do": do, "v": v}[name][300, 1, 5] = float(value)
    s = session(docs, 1, 4, 2, d)
    got = run(s, (q, k, v, do, b), STARTS, biased)
    s.device_status()  # an infinity is reported, as beyond the fp16 range
    rest = torch.ones(sum(docs), dtype=torch.bool)
    rest[256:384] = False
    for name, t in zip(NAMES[:5], got):
        if name == "lse":
            continue
        ref, err = want[name]
        within(t[rest.cuda()], {name: (ref[rest.numpy()], err[rest.numpy()])}, name)
    clean = run(s, x, STARTS, biased)  # nothing is left for the next call
    for name, t in zip(NAMES, clean):
        within(t, want, name)
    assert s.device_status() == 0
