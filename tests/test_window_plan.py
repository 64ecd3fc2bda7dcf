"""Windowed plans without a GPU: what a shard needs and receives, pairs, and the
device tables, whose tiles are walked here as the kernels walk them (every visible
pair in exactly one tile of the forward and of the backward, every row read is the
key it stands for), against the mask's definition. Refusals."""
import ctypes as C

import numpy as np
import pytest

import synth
from oracle import window as W

FAKE = C.c_void_p(1 << 24)
PIECES, SEGS, FTILES, FORDER, FSHARD, BTILES, BORDER, BSHARD, COPY = range(9)

CASES = [
    # documents, cp, policy, window, sinks
    (synth.doc_lengths(1), 2, "llama3", 128, 4),
    (synth.doc_lengths(1), 2, "hybrid", 100, 0),
    ([1, 127, 128, 129, 255, 256, 1, 1, 600, 2], 3, "perdoc", 64, 4),
    ([1, 127, 128, 129, 255, 256, 1, 1, 600, 2], 2, "perdoc", 1, 0),
    ([1, 127, 128, 129, 255, 256, 1, 1, 600, 2], 1, "perdoc", 1, 1),
    ([1200], 4, "perdoc", 128, 8),
    ([1200], 8, "perdoc", 300, 64),
    ([1201], 1, "perdoc", 5000, 4),
    ([700, 500], 2, "wholedoc", 129, 16),
    ([9, 20, 31, 40], 4, "perdoc", 3, 7),   # shards hold parts of the sinks
    ([40, 24], 8, "llama3", 2, 20),
    ([64] * 9 + [37], 3, "perdoc", 31, 33),
    ([2500, 3], 2, "perdoc", 700, 1),
    ([300] * 4, 2, "hybrid", 2 ** 31 - 1, 3),
]


def tables(plan, image):
    import context_document_masked_gb300.fcp as lib
    dp = lib.DevPlan()
    assert lib.raw_call("fcp_plan_bind", plan._ptr, FAKE, plan.device_bytes(), C.byref(dp)) == lib.OK
    width = {PIECES: 8, SEGS: 4, FTILES: 4, BTILES: 12, COPY: 4}
    out = {}
    for t in range(9):
        n = dp.counts[t] * width.get(t, 1)
        x = image[dp.tables[t]:dp.tables[t] + n]
        out[t] = x.reshape(-1, width[t]) if t in width else x
    return out


def mask(docs, window, sinks):
    T = sum(docs)
    m = np.zeros((T, T), bool)
    a = 0
    for n in docs:
        m[a:a + n, a:a + n] = W.visible(n, window, sinks)
        a += n
    return m


@pytest.mark.parametrize("docs,cp,policy,window,sinks", CASES)
def test_needs_and_pairs(lib, docs, cp, policy, window, sinks):
    base = lib.Plan(docs, cp, policy)
    p = base.windowed(window, sinks)
    off = np.concatenate([[0], np.cumsum(docs)])
    total, at = [], 0
    for j in range(cp):
        s, b = p.shard(j), base.shard(j)
        assert s["pieces"] == b["pieces"] and s["tokens"] == b["tokens"]
        need = W.needed_keys(docs, s["pieces"], window, sinks)
        got = np.zeros(sum(docs), int)
        for doc, x, y in s["kv_need"]:
            assert off[doc] <= x < y <= off[doc + 1]
            got[x:y] += 1
        assert np.array_equal(got, need.astype(int))
        own, recv = np.zeros(sum(docs), bool), np.zeros(sum(docs), int)
        for _, x, y in s["pieces"]:
            own[x:y] = True
        for _, x, y in s["kv_remote"]:
            recv[x:y] += 1
        assert recv.max(initial=0) <= 1 and (recv[need & ~own] == 1).all() and (recv[~need] == 0).all()
        assert [r[1] for r in s["kv_remote"]] == sorted(r[1] for r in s["kv_remote"])
        # A key of its own that a shard receives: a sink, of a document of which it holds a part of the sinks it needs.
        twice = np.flatnonzero((recv > 0) & own)
        for key in twice:
            o = off[np.searchsorted(off, key, side="right") - 1]
            outside = [k for k in range(o, o + sinks) if any(a <= q < e and q - k >= window for _, a, e in s["pieces"]
                                                              for q in range(max(a, o), e) if q < off[np.searchsorted(off, o, side="right")])]
            assert key in outside and not own[outside].all()
        assert s["remote_rows"] == recv.sum() and s["kbuf_base"] == at
        at += s["remote_rows"]
        assert s["useful_pairs"] == W.pairs(docs, s["pieces"], window, sinks)
        total.append(s["useful_pairs"])
    st = p.stats()
    assert st["total_pairs"] == sum(total) and st["max_pairs"] == max(total) and st["remote_rows_total"] == at
    assert st["imbalance"] == pytest.approx(max(total) / (sum(total) / cp), rel=1e-12)
    if window >= max(docs):
        assert at == base.stats()["remote_rows_total"] and st["total_pairs"] == base.stats()["total_pairs"]


def source_keys(t, rows):
    """The key in each received row."""
    key = np.full(max(rows, 1), -1)
    for src, dst, n, _ in t[COPY]:
        assert (key[dst:dst + n] == -1).all()
        key[dst:dst + n] = np.arange(src, src + n)
    assert rows == 0 or (key >= 0).all()
    return key


@pytest.mark.parametrize("docs,cp,policy,window,sinks", CASES)
def test_tables_cover_the_mask(lib, docs, cp, policy, window, sinks):
    p = lib.Plan(docs, cp, policy).windowed(window, sinks)
    t = tables(p, p.device_image())
    T, slots, W0 = sum(docs), (sinks + 7) // 8 * 8, min(window, sum(docs))
    rcv = source_keys(t, p.stats()["remote_rows_total"])
    want = mask(docs, window, sinks)

    def rows_of(src, row, n):
        assert row >= 0 and row + n <= (len(rcv) if src else T)
        return rcv[row:row + n] if src else np.arange(row, row + n)

    # Forward: a tile's queries against its walker's key tiles.
    seen, tiles, queries = np.zeros((T, T), int), 0, np.zeros(T, int)
    for piece, q0, qr, cost in t[FTILES]:
        _, _, start, end, ds, sb, sc, sink_row = t[PIECES][piece]
        assert start <= q0 and q0 + qr <= end and 1 <= qr <= 128
        queries[q0:q0 + qr] += 1
        q = np.arange(q0, q0 + qr)
        take = slots if q[-1] - W0 >= ds and sinks else 0
        n_tiles = 0
        if take:
            s = np.arange(ds, ds + sinks)
            hit = s <= q[:, None] - W0
            used = s[hit.any(0)]
            assert np.array_equal(rows_of(sink_row >= 0, sink_row if sink_row >= 0 else ds, len(used)), used)
            seen[np.ix_(q, used)] += hit[:, :len(used)]
        for src, row, ks, ln in t[SEGS][sb:sb + sc]:
            a, e = max(ks, q0 - W0 + 1), min(ks + ln, q[-1] + 1)
            while a < e:
                n = min(128 - take, e - a)
                take = 0
                key = np.arange(a, a + n)
                assert np.array_equal(rows_of(src, row + a - ks, n), key)
                seen[np.ix_(q, key)] += (key <= q[:, None]) & (q[:, None] - key < W0)
                a += n
                n_tiles += 1
        assert n_tiles == cost
        tiles += n_tiles
    assert (queries == 1).all() and np.array_equal(seen, want.astype(int))
    assert tiles == sum(p.shard(j)["fwd_tiles"] for j in range(cp))

    # Backward: a unit's key tile against its query tiles.
    seen = np.zeros((T, T), int)
    for key0, n, src, row, doc, sink_row, na, q0, q_end, nb, piece, _ in t[BTILES]:
        _, _, start, end, ds, _, _, piece_sinks = t[PIECES][piece]
        assert na == 0 and nb == -(-(q_end - q0) // 128) > 0 and start <= q0 < q_end <= end
        key = np.arange(key0, key0 + n)
        assert np.array_equal(rows_of(src, row, n), key)
        q = np.arange(q0, q_end)
        seen[np.ix_(q, key)] += (key <= q[:, None]) & (q[:, None] - key < W0)
        if doc < 0:
            assert n <= 128
            continue
        assert doc == ds and sink_row == piece_sinks and n <= 128 - slots
        for s in range(sinks):
            for i in range(max(key0, ds + s + W0), key0 + n):
                assert q0 <= i < q_end
                assert rows_of(sink_row >= 0, sink_row + s if sink_row >= 0 else ds + s, 1)[0] == ds + s
                seen[i, ds + s] += 1
    assert np.array_equal(seen, want.astype(int))
    assert sorted(t[FORDER]) == list(range(len(t[FTILES]))) and sorted(t[BORDER]) == list(range(len(t[BTILES])))


@pytest.mark.parametrize("docs,cp,policy,window,sinks", CASES)
def test_double_tiles_cover_the_mask(lib, docs, cp, policy, window, sinks):
    """The double query tiles (two runs of up to 128 rows of one head), walked as the forward walks them."""
    p = lib.Plan(docs, cp, policy).windowed(window, sinks)
    image = p.device_image()
    t = tables(p, image)
    dp = lib.DevPlan()
    assert lib.raw_call("fcp_plan_bind", p._ptr, FAKE, p.device_bytes(), C.byref(dp)) == lib.OK
    doubles = image[dp.tables[14]:dp.tables[14] + 4 * dp.counts[14]].reshape(-1, 4)
    shard = image[dp.tables[15]:dp.tables[15] + cp + 1]
    assert dp.counts[15] == cp + 1 and shard[0] == 0 and shard[-1] == len(doubles)
    T, slots, W0 = sum(docs), (sinks + 7) // 8 * 8, min(window, sum(docs))
    seen, queries = np.zeros((T, T), int), np.zeros(T, int)
    for j in range(cp):
        for piece, q0, first, second in doubles[shard[j]:shard[j + 1]]:
            owner, _, start, end, ds, sb, sc, _ = t[PIECES][piece]
            n = first + second
            assert owner == j and start <= q0 and q0 + n <= end and 1 <= first <= 128 and 0 <= second <= 128
            q = np.arange(q0, q0 + n)
            queries[q] += 1
            take = slots if q[-1] - W0 >= ds and sinks else 0
            for s in range(ds, ds + sinks if take else ds):
                seen[q[s <= q - W0], s] += 1
            for _, _, ks, ln in t[SEGS][sb:sb + sc]:
                key = np.arange(max(ks, q0 - W0 + 1), min(ks + ln, q[-1] + 1))
                seen[np.ix_(q, key)] += (key <= q[:, None]) & (q[:, None] - key < W0)
    assert (queries == 1).all() and np.array_equal(seen, mask(docs, window, sinks).astype(int))


def test_windows_of_a_plan_are_independent(lib):
    base = lib.Plan([1000, 200], 2, "perdoc")
    image = base.device_image()
    p = base.windowed(64, 4)
    again = p.windowed(300, 0)  # of a windowed plan: the same shards
    assert np.array_equal(again.device_image(), base.windowed(300, 0).device_image())
    assert np.array_equal(base.device_image(), image)
    w = p.device_image()
    del base
    assert np.array_equal(p.device_image(), w) and p.window == 64 and p.sinks == 4


def test_a_window_cuts_what_is_received(lib):
    """One document of 64K over eight shards: a window and the sinks before each of 15 pieces, not whole prefixes."""
    base = lib.Plan([65536], 8, "perdoc")
    assert base.windowed(2048, 4).stats()["remote_rows_total"] == 15 * 2047 - 2047 + 7 * 4


def test_refusals(lib):
    p = lib.Plan([100, 28], 1, "perdoc")
    out = C.c_void_p(5)
    for plan, window, sinks, st in ((None, 4, 0, lib.ERR_INVALID_ARG), (p._ptr, 0, 0, lib.ERR_INVALID_ARG),
                                    (p._ptr, -3, 0, lib.ERR_INVALID_ARG), (p._ptr, 4, -1, lib.ERR_INVALID_ARG),
                                    (p._ptr, 4, 65, lib.ERR_UNSUPPORTED)):
        assert lib.raw_call("fcp_plan_window", plan, window, sinks, C.byref(out)) == st
        assert out.value is None
    assert lib.raw_call("fcp_plan_window", p._ptr, 4, 0, None) == lib.ERR_INVALID_ARG
    with pytest.raises(lib.FcpError):
        p.windowed(0)
    w = p.windowed(32, 4)
    dp = lib.DevPlan()
    assert lib.raw_call("fcp_plan_bind", w._ptr, FAKE, w.device_bytes(), C.byref(dp)) == lib.OK
    dm, ws = lib.dims(128, 4, 2, 64), 1 << 40
    rel = lib.RelBias(FAKE, (C.c_int32 * 1)(0), 1)
    uns, d = lib.ERR_UNSUPPORTED, C.byref(dp)
    assert lib.raw_call("fcp_attn_fwd_bias", FAKE, FAKE, FAKE, FAKE, FAKE, C.byref(rel), d, -1, 0, 128, dm, 0, FAKE, FAKE,
                        FAKE, ws, None) == uns
    assert lib.raw_call("fcp_attn_bwd_bias", FAKE, FAKE, FAKE, FAKE, FAKE, C.byref(rel), FAKE, 1, FAKE, FAKE, d, -1, dm, FAKE,
                        FAKE, FAKE, C.c_void_p(1 << 25), FAKE, ws, None) == uns
    assert lib.raw_call("fcp_attn_fwd_ring", FAKE, FAKE, FAKE, d, -1, -1, dm, 0, FAKE, FAKE, FAKE, ws, None) == uns
    assert lib.raw_call("fcp_attn_fwd_qk8", FAKE, FAKE, FAKE, FAKE, FAKE, d, -1, 0, 128, dm, 0, FAKE, FAKE, FAKE, ws, None) == uns
    assert lib.raw_call("fcp_attn_fwd_noalloc", FAKE, FAKE, FAKE, FAKE, FAKE, d, -1, 0, 128, dm, 0, FAKE, FAKE, None) == uns
    # What a windowed plan serves is checked as ever.
    assert lib.raw_call("fcp_attn_fwd", FAKE, FAKE, FAKE, FAKE, FAKE, d, -1, 0, 129, dm, 0, FAKE, FAKE, FAKE, ws,
                        None) == lib.ERR_INVALID_ARG


def test_session_refuses_sinks_without_a_window(lib):
    pytest.importorskip("torch")
    from context_document_masked_gb300.session import CPAttention
    with pytest.raises(ValueError, match="window"):
        CPAttention([64], 1, "perdoc", 4, 2, 64, device="cpu", sinks=4)


def test_lengths_above_32_bits(lib):
    p = lib.Plan([300, 212], 2, "hybrid")
    whole = p.windowed(512, 4)
    for window in (2**31 - 1, 2**31, 2**32 + 1, 2**63):
        assert p.windowed(window, 4).stats() == whole.stats(), window
    for window, sinks in ((-2**32 + 8, 0), (-2**31 - 1, 0), (8, 2**32), (8, 2**32 + 4), (8, -2**32)):
        with pytest.raises(lib.FcpError):
            p.windowed(window, sinks)
