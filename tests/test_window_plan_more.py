"""Windowed plans without a GPU, more of them: the double query tiles with the rows that they read, and how many key
segments a piece has."""
import ctypes as C

import numpy as np
import pytest

from test_window_plan import CASES, FAKE, PIECES, SEGS, mask, source_keys, tables

POLICIES = ("llama3", "perdoc", "wholedoc", "hybrid", "hybrid_tiles")
MOST_SEGS = 6  # what the forward holds of a unit
# The last document ends before its sinks do, and is longer than the window.
SHORT_LAST = [([100, 20], 1, "perdoc", 8, 33), ([40, 30], 2, "perdoc", 4, 64), ([5, 9], 1, "wholedoc", 2, 64)]


@pytest.mark.parametrize("docs,cp,policy,window,sinks", CASES + SHORT_LAST)
def test_double_tiles_read_the_keys_they_stand_for(lib, docs, cp, policy, window, sinks):
    """Every visible pair in one key tile of one double tile, every row read (own, received, sinks) the key it stands for."""
    p = lib.Plan(docs, cp, policy).windowed(window, sinks)
    image = p.device_image()
    t = tables(p, image)
    dp = lib.DevPlan()
    assert lib.raw_call("fcp_plan_bind", p._ptr, FAKE, p.device_bytes(), C.byref(dp)) == lib.OK
    doubles = image[dp.tables[14]:dp.tables[14] + 4 * dp.counts[14]].reshape(-1, 4)
    shard = image[dp.tables[15]:dp.tables[15] + cp + 1]
    assert dp.counts[15] == cp + 1 and shard[0] == 0 and shard[-1] == len(doubles)
    T, slots, W0 = sum(docs), (sinks + 7) // 8 * 8, min(window, sum(docs))
    rcv = source_keys(t, p.stats()["remote_rows_total"])

    def rows_of(src, row, n):
        assert row >= 0 and row + n <= (len(rcv) if src else T)
        return rcv[row:row + n] if src else np.arange(row, row + n)

    seen, queries = np.zeros((T, T), int), np.zeros(T, int)
    for j in range(cp):
        for piece, q0, first, second in doubles[shard[j]:shard[j + 1]]:
            owner, doc, start, end, ds, sb, sc, sink_row = t[PIECES][piece]
            n = first + second
            assert owner == j and start <= q0 and q0 + n <= end and 1 <= first <= 128 and 0 <= second <= 128
            q = np.arange(q0, q0 + n)
            queries[q] += 1
            take = slots if q[-1] - W0 >= ds and sinks else 0
            if take:
                s = np.arange(ds, min(ds + sinks, ds + docs[doc]))
                hit = s <= q[:, None] - W0
                used = s[hit.any(0)]
                assert np.array_equal(rows_of(sink_row >= 0, sink_row if sink_row >= 0 else ds, len(used)), used)
                seen[np.ix_(q, used)] += hit[:, :len(used)]
            for src, row, ks, ln in t[SEGS][sb:sb + sc]:
                a, e = max(ks, q0 - W0 + 1), min(ks + ln, q[-1] + 1)
                while a < e:
                    m = min(128 - take, e - a)
                    take = 0
                    key = np.arange(a, a + m)
                    assert np.array_equal(rows_of(src, row + a - ks, m), key)
                    seen[np.ix_(q, key)] += (key <= q[:, None]) & (q[:, None] - key < W0)
                    a += m
    assert (queries == 1).all() and np.array_equal(seen, mask(docs, window, sinks).astype(int))


def test_segments_of_a_piece(lib):
    """At most as many as the forward holds of a unit, under every policy, windows and sinks of all lengths among them."""
    rng = np.random.default_rng(17)
    most = 0
    for _ in range(1500):
        cp = int(rng.integers(1, 17))
        docs = [int(x) for x in rng.integers(1, int(rng.choice([3, 12, 60, 400])), int(rng.integers(1, 12)))]
        docs[-1] += -sum(docs) % (2 * cp)  # what every policy can shard
        p = lib.Plan(docs, cp, str(rng.choice(POLICIES)))
        sinks = int(rng.integers(0, 65))
        w = p.windowed(int(2 ** rng.uniform(0, 9)), sinks)
        pieces = tables(w, w.device_image())[PIECES]
        most = max(most, int(pieces[:, 6].max()))
        for j in range(cp):
            doc = [x[0] for x in w.shard(j)["pieces"]]
            assert all(doc.count(x) <= 2 for x in doc)
    assert 4 <= most <= MOST_SEGS
