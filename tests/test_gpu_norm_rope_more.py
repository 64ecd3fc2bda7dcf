"""More of the head norm and rotation's gradient: calls that share what they add to."""
import pytest
import torch

from test_gpu_norm_rope import make, session, slices

pytestmark = pytest.mark.gpu


def test_two_calls_add_to_one_gradient(cuda):
    """Micro-batches in two sessions on two streams, adding to one dwq and dwk: what
    each gives alone, as often as it was called."""
    docs, hq, hkv, d, rounds = [300, 1, 83], 6, 2, 64, 64
    runs = []
    for n in range(2):
        qkv, w, f, g = make(docs, hq, hkv, d, d, seed=90 + n)
        s, x = session(docs, 2, hq, hkv, d), qkv.cuda()
        args = (*(t.cuda() for t in g), *slices(x, hq, hkv)[:2])
        kw = dict(wq=w[0].cuda(), wk=w[1].cuda(), inv_freq=f.cuda())
        own = s.qk_norm_rope_backward(*args, **kw)
        runs.append((s, args, dict(kw, dq_in=own[0], dk_in=own[1], dv_in=own[2]), own[3:], torch.cuda.Stream()))
    sums = [torch.zeros(d, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(rounds):
        for s, args, kw, _own, st in runs:
            with torch.cuda.stream(st):
                s.qk_norm_rope_backward(*args, **kw, dwq=sums[0], dwk=sums[1])
    torch.cuda.synchronize()
    for i, t in enumerate(sums):
        a, b = (r[3][i].double() for r in runs)
        # 2 rounds additions of equal terms in some order, each off by half a step of a sum no larger than all terms.
        tol = 2 * rounds * 2.0 ** -24 * rounds * (a.abs() + b.abs())
        assert ((t.double() - rounds * (a + b)).abs() <= tol).all()
        assert (torch.minimum(a.abs(), b.abs()) > tol).double().mean() > 0.9  # one call's share would be missed


def test_given_weight_gradients_added_to_or_written(cuda):
    docs, hq, hkv, d = [300, 1, 83], 6, 2, 64
    qkv, w, f, g = make(docs, hq, hkv, d, d, seed=92)
    s, x = session(docs, 2, hq, hkv, d), qkv.cuda()
    args = (*(t.cuda() for t in g), *slices(x, hq, hkv)[:2])
    kw = dict(wq=w[0].cuda(), wk=w[1].cuda(), inv_freq=f.cuda())
    alone = s.qk_norm_rope_backward(*args, **kw)[3:]
    dw = [torch.full((d,), float("nan"), device="cuda") for _ in range(2)]
    got = s.qk_norm_rope_backward(*args, **kw, dwq=dw[0], dwk=dw[1], zero_grads=True)[3:]
    assert got[0] is dw[0] and got[1] is dw[1] and torch.equal(dw[0], alone[0]) and torch.equal(dw[1], alone[1])
    s.qk_norm_rope_backward(*args, **kw, dwq=dw[0], dwk=dw[1])
    assert torch.equal(dw[0], 2 * alone[0]) and torch.equal(dw[1], 2 * alone[1])
    one = torch.full((d,), float("nan"), device="cuda")
    got = s.qk_norm_rope_backward(*args, **kw, dwk=one, zero_grads=True)[3:]
    assert got[1] is one and torch.equal(got[0], alone[0]) and torch.equal(one, alone[1])


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("rot", [0, 32])
def test_infinities_in_dimensions_that_pass(cuda, rot, inter):
    """Rotation alone: a dimension that does not turn passes whatever it holds, and no
    other one sees it; the same for the gradient."""
    docs, hq, hkv, d = [40, 1, 23], 3, 1, 64
    qkv, _, f, _ = make(docs, hq, hkv, d, rot, seed=93)
    s, x = session(docs, 2, hq, hkv, d), qkv.cuda()
    kw = dict(inv_freq=f.cuda() if rot else None, norm=False, interleaved=inter)
    plain = s.qk_norm_rope(*slices(x, hq, hkv), **kw)
    bad = x.clone()
    at = [rot, rot + 5, 63]
    bad[3, 1, at[0]], bad[20, 3, at[1]], bad[50, 2, at[2]] = float("inf"), float("nan"), float("-inf")
    got = s.qk_norm_rope(*slices(bad, hq, hkv), **kw)
    for a, b, xin, xbad in zip(plain, got, slices(x, hq, hkv), slices(bad, hq, hkv)):
        hit = ~torch.isfinite(xbad)
        assert torch.equal(a[~hit], b[~hit])
        assert torch.allclose(b[hit], xbad[hit], rtol=0, atol=0, equal_nan=True)  # infinities with their sign, NaN as NaN
    g = [t.float() for t in plain[:2]]
    gbad = [t.clone() for t in g]
    gbad[0][3, 1, at[0]], gbad[1][50, 0, at[2]] = float("inf"), float("nan")
    a = s.qk_norm_rope_backward(*g, None, None, None, **kw)[:2]
    b = s.qk_norm_rope_backward(*gbad, None, None, None, **kw)[:2]
    for m, n, t in zip(a, b, gbad):
        hit = ~torch.isfinite(t)
        assert hit.sum() == 1 and torch.equal(m[~hit], n[~hit]) and not torch.isfinite(n[hit]).any()
