"""More of the attention with a bucketed distance bias: bucket starts at the
type's end, sums that several calls share, long documents in closed form.

Bounds as derived in test_gpu_rel_bias."""
import pytest
import torch

from test_gpu_rel_bias import make, reference, session, step, within

pytestmark = pytest.mark.gpu

NAMES = ("out", "lse", "dq", "dk", "dv", "dbias")
LAST = 2 ** 31 - 1


@pytest.mark.parametrize("starts", [[0, 5, LAST], [0, LAST - 40, LAST - 31, LAST - 30, LAST - 1, LAST, LAST],
                                    [0, 1, 8191, 8192, 8193, 8447, 8448, LAST - 255]], ids=["end", "near", "table"])
def test_starts_at_the_end_of_the_type(cuda, starts):
    """Buckets that no distance of the sequence reaches get no gradient, wherever they start."""
    docs, hq, hkv, d = [300, 1, 83], 4, 2, 64
    x = make(docs, hq, hkv, d, len(starts), seed=11)
    want = reference(*x, starts, docs)
    s = session(docs, 2, hq, hkv, d)
    got = step(s, [t.cuda() for t in x], starts)
    for name, t in zip(NAMES, got):
        within(t, want, name)
    beyond = [u for u, first in enumerate(starts) if first >= 300]
    assert (got[5][:, beyond] == 0).all() and s.device_status() == 0


def test_two_calls_add_to_one_gradient(cuda):
    """Micro-batches in two sessions on two streams, all adding to one dk, dv and dbias:
    what each adds alone, as often as it was called."""
    from context_document_masked_gb300 import fcp
    docs, hq, hkv, d, rounds = [700, 1, 323], 4, 2, 64, 16
    starts, T = fcp.rel_buckets(32, 128), sum(docs)
    runs = []
    for n in range(2):
        x = make(docs, hq, hkv, d, 32, seed=80 + n)
        s, (q, k, v, do, b) = session(docs, 2, hq, hkv, d), [t.cuda() for t in x]
        s.gather(k, v)
        out, lse = s.forward_bias(q, k, v, b, starts, out_dtype=torch.float32)
        alone = s.backward_bias(q, k, v, out, lse, do, b, starts)
        runs.append((s, (q, k, v, out, lse, do, b, starts), alone, reference(*x, starts, docs), torch.cuda.Stream()))
    sums = [torch.zeros(T, hkv, d, device="cuda"), torch.zeros(T, hkv, d, device="cuda"), torch.zeros(hq, 32, device="cuda")]
    torch.cuda.synchronize()
    for _ in range(rounds):
        for s, x, alone, _w, st in runs:
            with torch.cuda.stream(st):
                s.backward_bias(*x, dq=alone[0], dk=sums[0], dv=sums[1], dbias=sums[2], zero_grads=False)
    torch.cuda.synchronize()
    for i, name in enumerate(("dk", "dv", "dbias")):
        # The terms are the same, their order is not. A term goes through n additions at most, each off by 2^-24 of a
        # partial sum: 64 along its diagonal, 64 tiles that share a distance, 40 distances and lanes of a bucket, and
        # the two sessions' rounds. The terms' sizes are at most 2^11 / 3 of a call's bound, which has 3 2^-11 of them.
        n = 64 + 64 + 40 + 2 * rounds
        ref = rounds * sum(r[2][i + 1].double().cpu() for r in runs)
        size = sum(torch.from_numpy(r[3][name][1]) for r in runs) * 2.0 ** 11 / 3
        tol = rounds * n * 2.0 ** -24 * size
        assert ((sums[i].double().cpu() - ref).abs() <= tol).all(), name
        if name == "dbias":  # a call's share would be missed in most buckets
            assert ((torch.minimum(*(r[2][3].double().cpu().abs() for r in runs)) > tol).double().mean() > 0.5)


def test_one_shard_into_given_gradients_says_how(cuda):
    """A loop over shards must not keep the last one's share by a default."""
    docs, hq, hkv, d, starts = [300, 84], 4, 2, 64, [0, 1, 50]
    x = make(docs, hq, hkv, d, 3, seed=12)
    want = reference(*x, starts, docs)
    q, k, v, do, b = (t.cuda() for t in x)
    s = session(docs, 2, hq, hkv, d)
    s.gather(k, v)
    out, lse = s.forward_bias(q, k, v, b, starts, out_dtype=torch.float32)
    T, nan = sum(docs), float("nan")
    g = dict(dq=torch.empty(T, hq, d, device="cuda"), dk=torch.full((T, hkv, d), nan, device="cuda"),
             dv=torch.full((T, hkv, d), nan, device="cuda"), dbias=torch.full((hq, 3), nan, device="cuda"))
    for name in ("dk", "dv", "dbias"):
        with pytest.raises(ValueError, match="zero_grads"):
            s.backward_bias(q, k, v, out, lse, do, b, starts, shard=0, **{name: g[name]})
        assert g[name].isnan().all()
    for j in range(2):
        s.gather(k, v, shard=j)
        s.backward_bias(q, k, v, out, lse, do, b, starts, shard=j, zero_grads=j == 0, **g)
    for name, t in g.items():
        within(t, want, name)
    s.gather(k, v, shard=1)
    new = s.backward_bias(q, k, v, out, lse, do, b, starts, shard=1)[1:]  # new ones start from zero
    s.backward_bias(q, k, v, out, lse, do, b, starts, shard=1, zero_grads=True, **g)
    for a, t in zip(new, (g["dk"], g["dv"], g["dbias"])):
        assert torch.allclose(a, t, rtol=0, atol=1e-5)
