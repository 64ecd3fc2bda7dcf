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
