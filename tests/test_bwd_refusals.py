"""Argument checks of the backward that come before any launch, on the CPU (the
device pointers below are never dereferenced)."""
import ctypes as C

import pytest

import synth


def at(k, off=0):
    return C.c_void_p((1 << 24) * (k + 1) + off)


@pytest.fixture()
def bound(lib):
    docs = synth.doc_lengths(1)
    p = lib.Plan(docs, 2, "perdoc")
    dp = lib.DevPlan()
    assert lib.raw_call("fcp_plan_bind", p._ptr, at(0), p.device_bytes(), C.byref(dp)) == lib.OK
    assert all(p.shard(j)["remote_rows"] > 0 for j in range(2))
    return p, dp, lib.dims(sum(docs), 4, 2, 64)


def backward(lib, dp, dm, shard, kbuf, vbuf, biased):
    ws_bytes = 1 << 40
    if not biased:
        return lib.raw_call("fcp_attn_bwd", at(1), at(2), at(3), kbuf, vbuf, at(6), 1, at(7), at(8), C.byref(dp), shard, dm,
                            at(9), at(10), at(11), at(12), ws_bytes, None)
    starts = (C.c_int32 * 2)(0, 1)
    rb = lib.RelBias(at(13), starts, 2, 0)
    return lib.raw_call("fcp_attn_bwd_bias", at(1), at(2), at(3), kbuf, vbuf, C.byref(rb), at(6), 1, at(7), at(8),
                        C.byref(dp), shard, dm, at(9), at(10), at(11), at(14), at(12), ws_bytes, None)


@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
@pytest.mark.parametrize("shard", [-1, 0, 1])
def test_received_keys_are_aligned(lib, bound, shard, biased):
    """Like every device pointer, in steps of 16 bytes: both are read 16 bytes at a time."""
    p, dp, dm = bound
    for off in (2, 4, 8):
        assert backward(lib, dp, dm, shard, at(4, off), at(5), biased) == lib.ERR_INVALID_ARG
        assert backward(lib, dp, dm, shard, at(4), at(5, off), biased) == lib.ERR_INVALID_ARG
    for kbuf, vbuf in ((None, at(5)), (at(4), None)):
        assert backward(lib, dp, dm, shard, kbuf, vbuf, biased) == lib.ERR_INVALID_ARG
