"""Argument checks of the bucketed distance bias, on the CPU: every refusal
comes from the host checks, before any launch (the device pointers below are
never dereferenced). The bucket helper against its formula."""
import ctypes as C
from decimal import ROUND_FLOOR, Decimal, getcontext

import numpy as np
import pytest

import synth

torch = pytest.importorskip("torch")

FAKE, FAKE_GRAD = C.c_void_p(1 << 24), C.c_void_p(1 << 25)


@pytest.fixture()
def bound(lib):
    docs = synth.doc_lengths(1)
    p = lib.Plan(docs, 2, "hybrid")
    dp = lib.DevPlan()
    assert lib.raw_call("fcp_plan_bind", p._ptr, FAKE, p.device_bytes(), C.byref(dp)) == lib.OK
    return p, dp, lib.dims(sum(docs), 4, 2, 64)


def rel(lib, starts, bias=FAKE, n=None):
    a = (C.c_int32 * max(1, len(starts)))(*starts)
    return lib.RelBias(bias, a if starts else None, len(starts) if n is None else n)


def calls(lib, dp, dm, rb, dbias=FAKE_GRAD, ws_bytes=1 << 40):
    r = C.byref(rb) if rb is not None else None
    return (lib.raw_call("fcp_attn_fwd_bias", FAKE, FAKE, FAKE, FAKE, FAKE, r, C.byref(dp), -1, 0, dm.T, dm, 0, FAKE, FAKE,
                         FAKE, ws_bytes, None),
            lib.raw_call("fcp_attn_bwd_bias", FAKE, FAKE, FAKE, FAKE, FAKE, r, FAKE, 1, FAKE, FAKE, C.byref(dp), -1, dm,
                         FAKE, FAKE, FAKE, dbias, FAKE, ws_bytes, None))


def test_bias_table_and_starts(lib, bound):
    p, dp, dm = bound
    inv, uns = lib.ERR_INVALID_ARG, lib.ERR_UNSUPPORTED
    for rb, st in ((None, inv), (rel(lib, [0, 1], bias=None), inv), (rel(lib, [0, 1], bias=C.c_void_p((1 << 24) + 2)), inv),
                   (rel(lib, []), inv), (rel(lib, [0, 1], n=0), inv), (rel(lib, [0, 1], n=-3), inv), (rel(lib, [1, 2]), inv),
                   (rel(lib, [-1, 2]), inv), (rel(lib, [0, 5, 4]), inv), (rel(lib, list(range(129))), uns)):
        assert calls(lib, dp, dm, rb) == (st, st)
    for flag in (-1, 2):
        rb = rel(lib, [0, 1])
        rb.zero_grads = flag
        assert calls(lib, dp, dm, rb) == (inv, inv)
    good = rel(lib, [0, 0, 7])
    assert calls(lib, dp, dm, good, dbias=None)[1] == inv
    assert calls(lib, dp, dm, good, dbias=C.c_void_p((1 << 24) + 1))[1] == inv
    for off in (0, -44, 44):  # the gradient inside the table of 4 x 3
        assert calls(lib, dp, dm, good, dbias=C.c_void_p((1 << 24) + off))[1] == inv
    for off in (-48, 48):
        assert calls(lib, dp, dm, good, dbias=C.c_void_p((1 << 24) + off), ws_bytes=1024)[1] == lib.ERR_CAPACITY
    assert calls(lib, dp, dm, good, ws_bytes=1024) == (lib.ERR_CAPACITY, lib.ERR_CAPACITY)
    assert calls(lib, dp, lib.dims(dm.T, 4, 2, 96), good) == (uns, uns)
    assert calls(lib, dp, lib.dims(dm.T, 4, 3, 64), good) == (uns, uns)
    assert calls(lib, dp, lib.dims(dm.T, 4, 2, 64, 1e-31), good) == (uns, uns)
    dp.counts[2] += 1
    assert calls(lib, dp, dm, good) == (inv, inv)


def test_binding_checks_on_host_tensors(lib, bound):
    p, dp, dm = bound
    dplan = lib.DevicePlan(dp, p, None)
    q, k = torch.zeros(dm.T, 4, 64, dtype=torch.bfloat16), torch.zeros(dm.T, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        lib.attn_fwd_bias(q, k, k, k, k, torch.zeros(4, 2), [0, 1], dplan, -1, q, torch.zeros(4, dm.T), torch.zeros(4))
    for starts in ([], [[0, 1]], [0.0, 1.0], [0, 1 << 31], [-1, 3]):
        with pytest.raises(ValueError, match="starts"):
            lib._rel_bias(torch.zeros(4, 2), starts, 4)


@pytest.mark.parametrize("n,reach", [(2, 5), (8, 64), (17, 934), (32, 128), (48, 2000), (64, 8192), (128, 200), (33, 100)])
def test_bucket_starts(lib, n, reach):
    """Every distance's bucket, by logarithms of 50 digits."""
    getcontext().prec = 50
    starts, exact = lib.rel_buckets(n, reach), n // 2
    assert starts.dtype == np.int32 and starts[0] == 0 and (np.diff(starts) >= 0).all()
    for x in list(range(reach + 3)) + [10 * reach]:
        b = x
        if x >= exact:
            f = Decimal(n - exact) * (Decimal(x) / exact).ln() / (Decimal(reach) / exact).ln()
            b = min(n - 1, exact + int((f + Decimal("1e-30")).to_integral_value(rounding=ROUND_FLOOR)))
        assert (starts <= x).sum() - 1 == b, x


def test_bucket_starts_refusals(lib):
    out = (C.c_int32 * 200)()
    assert lib.raw_call("fcp_rel_buckets", 32, 128, None) == lib.ERR_INVALID_ARG
    assert lib.raw_call("fcp_rel_buckets", 1, 128, out) == lib.ERR_INVALID_ARG
    assert lib.raw_call("fcp_rel_buckets", 32, 16, out) == lib.ERR_INVALID_ARG
    assert lib.raw_call("fcp_rel_buckets", 129, 1000, out) == lib.ERR_UNSUPPORTED
    with pytest.raises(lib.FcpError):
        lib.rel_buckets(0, 10)
