"""Argument checks of the head norm and rotation, on the CPU: every refusal
comes from the host checks, before any launch (the device pointers below are
never dereferenced)."""
import ctypes as C

import pytest

import synth

torch = pytest.importorskip("torch")

HQ, HKV, D = 4, 2, 128
FUSED = (HQ + 2 * HKV) * D
BASE = 1 << 30
SPAN = 1 << 24


def at(i, off=0):
    return C.c_void_p(BASE + i * SPAN + off)


@pytest.fixture()
def bound(lib):
    docs = synth.doc_lengths(1)
    p = lib.Plan(docs, 2, "hybrid")
    dp = lib.DevPlan()
    assert lib.raw_call("fcp_plan_bind", p._ptr, at(0), p.device_bytes(), C.byref(dp)) == lib.OK
    return p, dp, sum(docs)


def fwd(lib, dp, T, **over):
    a = dict(q_in=at(1), sq=FUSED, k_in=at(1, HQ * D * 2), sk=FUSED, v_in=at(1, (HQ + HKV) * D * 2), sv=FUSED, wq=at(2),
             wk=at(2, 512), f=at(2, 1024), nr=lib.NormRope(1, 1e-6, D, 0, 1), shard=-1, dims=lib.dims(T, HQ, HKV, D),
             q=at(3), k=at(4), v=at(5))
    a.update(over)
    return lib.raw_call("fcp_qk_norm_rope", a["q_in"], a["sq"], a["k_in"], a["sk"], a["v_in"], a["sv"], a["wq"], a["wk"],
                        a["f"], C.byref(a["nr"]) if a["nr"] else None, C.byref(dp), a["shard"], a["dims"], a["q"], a["k"],
                        a["v"], None)


def bwd(lib, dp, T, **over):
    a = dict(dq=at(1), dk=at(2), dv=at(3), q_in=at(4), sq=FUSED, k_in=at(4, HQ * D * 2), sk=FUSED, wq=at(5), wk=at(5, 512),
             f=at(5, 1024), nr=lib.NormRope(1, 1e-6, D, 0, 1), shard=-1, dims=lib.dims(T, HQ, HKV, D), dq_in=at(6), so=FUSED,
             dk_in=at(6, HQ * D * 2), dv_in=at(6, (HQ + HKV) * D * 2), dwq=at(7), dwk=at(7, 512), ws=at(8), ws_bytes=1 << 40)
    a.update(over)
    return lib.raw_call("fcp_qk_norm_rope_bwd", a["dq"], a["dk"], a["dv"], a["q_in"], a["sq"], a["k_in"], a["sk"], a["wq"],
                        a["wk"], a["f"], C.byref(a["nr"]) if a["nr"] else None, C.byref(dp), a["shard"], a["dims"],
                        a["dq_in"], a["so"], a["dk_in"], a["so"], a["dv_in"], a["so"], a["dwq"], a["dwk"], a["ws"],
                        a["ws_bytes"], None)


def options(lib):
    N = lib.NormRope
    inv, uns = lib.ERR_INVALID_ARG, lib.ERR_UNSUPPORTED
    return {
        "no options": (dict(nr=None), inv), "norm 2": (dict(nr=N(2, 1e-6, D, 0, 1)), inv),
        "negative eps": (dict(nr=N(1, -1e-6, D, 0, 1)), inv), "nan eps": (dict(nr=N(1, float("nan"), D, 0, 1)), inv),
        "inf eps": (dict(nr=N(1, float("inf"), D, 0, 1)), inv), "rot over d": (dict(nr=N(1, 1e-6, D + 16, 0, 1)), inv),
        "rot negative": (dict(nr=N(1, 1e-6, -16, 0, 1)), inv), "rot 8": (dict(nr=N(1, 1e-6, 8, 0, 1)), uns),
        "pair order": (dict(nr=N(1, 1e-6, D, 2, 1)), inv), "weight type": (dict(nr=N(1, 1e-6, D, 0, 2)), inv),
        "add_dw 2": (dict(nr=N(1, 1e-6, D, 0, 1, 2)), inv),
        "no frequencies": (dict(f=None), inv), "misaligned frequencies": (dict(f=at(9, 2)), inv),
        "misaligned weights": (dict(wq=at(9, 2)), inv), "shard": (dict(shard=2), inv),
        "d 96": (dict(dims=lib.dims(2048, HQ, HKV, 96)), uns), "groups": (dict(dims=lib.dims(2048, 5, 2, D)), uns),
        "tokens": (dict(dims=lib.dims(2047, HQ, HKV, D)), inv),
        "no q_in": (dict(q_in=None), inv), "q_in misaligned": (dict(q_in=at(1, 8)), inv),
        "short stride": (dict(sq=HQ * D - 8), inv), "odd stride": (dict(sk=FUSED + 4), inv),
    }


@pytest.mark.parametrize("what", sorted(["no options", "norm 2", "negative eps", "nan eps", "inf eps", "rot over d",
                                         "rot negative", "rot 8", "pair order", "weight type", "add_dw 2", "no frequencies",
                                         "misaligned frequencies", "misaligned weights", "shard", "d 96", "groups", "tokens",
                                         "no q_in", "q_in misaligned", "short stride", "odd stride"]))
def test_options_and_inputs(lib, bound, what):
    p, dp, T = bound
    over, status = options(lib)[what]
    assert fwd(lib, dp, T, **over) == status
    assert bwd(lib, dp, T, **over) == status


def test_weights_need_the_norm(lib, bound):
    p, dp, T = bound
    nr = lib.NormRope(0, 0.0, D, 0, 1)
    assert fwd(lib, dp, T, nr=nr) == lib.ERR_INVALID_ARG
    assert bwd(lib, dp, T, nr=nr, wq=None, wk=None) == lib.ERR_INVALID_ARG        # dwq without a norm


def test_overlaps(lib, bound):
    p, dp, T = bound
    row = HQ * D * 2
    inv = lib.ERR_INVALID_ARG
    assert fwd(lib, dp, T, q=at(1)) == inv                                      # contiguous over the fused rows
    assert fwd(lib, dp, T, q_in=at(3, 16), sq=HQ * D) == inv                      # shifted by eight values
    assert fwd(lib, dp, T, q_in=at(3), sq=HQ * D + 8) == inv                      # other stride
    assert fwd(lib, dp, T, k=at(3, (T - 1) * row)) == inv                       # K over Q's last row
    assert fwd(lib, dp, T, v=None) == inv and fwd(lib, dp, T, v_in=None) == inv
    assert bwd(lib, dp, T, dq_in=at(1), so=HQ * D) == inv                         # over dq
    assert bwd(lib, dp, T, dk_in=at(6, HQ * D * 2 - 16)) == inv                   # slices of one row that share values
    assert bwd(lib, dp, T, dq_in=at(4, 16)) == inv
    assert bwd(lib, dp, T, dwk=at(7)) == inv and bwd(lib, dp, T, dwk=at(7, D * 4 - 4)) == inv   # one gradient over the other
    assert bwd(lib, dp, T, dv=None) == inv and bwd(lib, dp, T, dv_in=None) == inv


def test_workspace(lib, bound):
    p, dp, T = bound
    need = lib.workspace_bytes(lib.dims(T, HQ, HKV, D), p)
    assert bwd(lib, dp, T, ws=None) == lib.ERR_INVALID_ARG
    assert bwd(lib, dp, T, ws_bytes=need - 1) == lib.ERR_CAPACITY


def test_binding_refuses_host_tensors_and_shapes(lib, bound):
    p, dp, T = bound
    dplan = lib.DevicePlan(dp, p, None)
    x = torch.zeros(T, HQ, D, dtype=torch.bfloat16)
    y = torch.zeros(T, HKV, D, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        lib.qk_norm_rope(x, y, y, dplan, -1, x, y, y)
    g, h = x.float(), y.float()
    with pytest.raises(ValueError, match="CUDA tensor"):
        lib.qk_norm_rope_bwd(g, h, h, x, y, dplan, -1, x, y, y, None, None, torch.zeros(4))
