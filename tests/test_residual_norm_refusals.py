"""Argument checks of the residual norm, on the CPU: every refusal comes from
the host checks, before any launch (the device pointers below are never
dereferenced)."""
import ctypes as C

import pytest

import synth

torch = pytest.importorskip("torch")

STEP = 1 << 30  # between operands


@pytest.fixture()
def bound(lib):
    p = lib.Plan([48, 16], 2, "hybrid")
    dp = lib.DevPlan()
    assert lib.raw_call("fcp_plan_bind", p._ptr, C.c_void_p(1 << 24), p.device_bytes(), C.byref(dp)) == lib.OK
    return p, dp


def forward(lib, dp, n=64, rn=None, shard=-1, **kw):
    a = dict(x=1, y=2, gate=3, w_post=4, w_pre=5, x_out=6, h=7)
    a = {k: C.c_void_p(STEP * v) for k, v in a.items()}
    a.update({k: (None if v is None else C.c_void_p(v)) for k, v in kw.items() if not k.startswith("s_")})
    s = {k: kw.get("s_" + k, max(n, 8)) for k in a}
    rn = rn or lib.ResNorm(1, 1, 1, 1e-6, 1.0, 1.0, 0, 1, 0)
    return lib.raw_call("fcp_residual_norm", a["x"], s["x"], a["y"], s["y"], a["gate"], s["gate"], a["w_post"], a["w_pre"],
                        C.byref(rn), C.byref(dp), shard, n, a["x_out"], s["x_out"], a["h"], s["h"], None)


def backward(lib, dp, n=64, rn=None, shard=-1, ws_bytes=0, **kw):
    """With too small a workspace: ERR_CAPACITY stands for a call whose arguments pass."""
    names = "dh dx_out x_out y gate w_post w_pre dx dy dgate dw_post dw_pre ws".split()
    a = {k: C.c_void_p(STEP * (i + 1)) for i, k in enumerate(names)}
    a.update({k: (None if v is None else C.c_void_p(v)) for k, v in kw.items() if not k.startswith("s_")})
    s = {k: kw.get("s_" + k, max(n, 8)) for k in a}
    rn = rn or lib.ResNorm(1, 1, 1, 1e-6, 1.0, 1.0, 0, 1, 0)
    rows = [x for k in ("dh", "dx_out", "x_out", "y", "gate") for x in (a[k], s[k])]
    outs = [x for k in ("dx", "dy", "dgate") for x in (a[k], s[k])]
    return lib.raw_call("fcp_residual_norm_bwd", *rows, a["w_post"], a["w_pre"], C.byref(rn), C.byref(dp), shard, n, *outs,
                        a["dw_post"], a["dw_pre"], a["ws"], ws_bytes, None)


def test_sizes_and_options(lib, bound):
    _, dp = bound
    inv, uns, cap = lib.ERR_INVALID_ARG, lib.ERR_UNSUPPORTED, lib.ERR_CAPACITY
    for n in (0, -8, 4, 12, 16392):
        assert forward(lib, dp, n=n) == backward(lib, dp, n=n) == uns
        assert lib.residual_norm_ws_bytes(n) == 0
    for n in (8, 64, 16384):
        assert backward(lib, dp, n=n) == cap and lib.residual_norm_ws_bytes(n) >= 8 * n
    good = (1, 1, 1, 1e-6, 1.0, 1.0, 0, 1, 0)
    for i, bad in ((0, 2), (0, -1), (1, 2), (2, 2), (2, -1), (3, -1e-9), (3, float("inf")), (3, float("nan")),
                   (4, float("inf")), (5, float("nan")), (6, 2), (7, -1), (8, 5)):
        rn = lib.ResNorm(*good[:i], bad, *good[i + 1:])
        assert forward(lib, dp, rn=rn) == backward(lib, dp, rn=rn) == inv, (i, bad)
    for shard in (-2, 2):
        assert forward(lib, dp, shard=shard) == backward(lib, dp, shard=shard) == inv
    dp.counts[10] += 1
    assert forward(lib, dp) == backward(lib, dp) == inv


def test_pointers_strides_and_missing_parts(lib, bound):
    _, dp = bound
    inv, cap = lib.ERR_INVALID_ARG, lib.ERR_CAPACITY
    for k in ("x", "x_out", "h"):
        assert forward(lib, dp, **{k: None}) == inv
    for k in ("x", "y", "gate", "x_out", "h", "w_post", "w_pre"):
        assert forward(lib, dp, **{k: STEP * 9 + 8}) == inv, k
    for k in ("x", "y", "gate", "x_out", "h"):
        for stride in (56, 68, 0, -64, 1 << 62):
            assert forward(lib, dp, **{"s_" + k: stride}) == inv, (k, stride)
    assert forward(lib, dp, y=None) == forward(lib, dp, y=None, gate=None) == inv       # a gate, weights of no block
    assert forward(lib, dp, y=None, gate=None, w_post=None, x_out=None, h=None) == inv  # nothing to do
    rn = lib.ResNorm(1, 1, 1, 1e-6, 0.5, 1.0, 0, 1, 0)
    assert forward(lib, dp, rn=rn, y=None, gate=None, w_post=None, x_out=None) == inv   # a scaled residual has to be stored
    off = lib.ResNorm(1, 0, 1, 1e-6, 1.0, 1.0, 0, 1, 0)
    assert forward(lib, dp, rn=off) == forward(lib, dp, rn=off, h=None) == inv          # h, w_pre without the norm
    for k in ("dh", "x_out", "dx", "dy", "dgate"):
        assert backward(lib, dp, **{k: None}) == inv, k
    for k in ("dh", "dx_out", "x_out", "y", "gate", "dx", "dy", "dgate", "w_post", "w_pre", "ws"):
        assert backward(lib, dp, **{k: STEP * 19 + 8}) == inv, k
    for k in ("dw_post", "dw_pre"):
        assert backward(lib, dp, **{k: STEP * 19 + 2}) == inv, k
    for k in ("dh", "dx_out", "x_out", "y", "gate", "dx", "dy", "dgate"):
        for stride in (56, 68):
            assert backward(lib, dp, **{"s_" + k: stride}) == inv, (k, stride)
    assert backward(lib, dp, ws=None) == inv
    assert backward(lib, dp, dx_out=None) == backward(lib, dp, gate=None, dgate=None) == cap
    assert backward(lib, dp, y=None, gate=None, w_post=None, dy=None, dgate=None) == inv  # dw_post without a block
    assert backward(lib, dp, y=None, gate=None, w_post=None, dy=None, dgate=None, dw_post=None) == cap
    assert backward(lib, dp, rn=off) == inv
    assert backward(lib, dp, rn=off, dh=None, w_pre=None) == inv                        # dw_pre without the norm
    assert backward(lib, dp, rn=off, dh=None, w_pre=None, dw_pre=None, x_out=None) == cap
    assert backward(lib, dp, rn=off, dh=None, w_pre=None, dw_pre=None, dx_out=None) == inv


def test_overlaps(lib, bound):
    _, dp = bound
    inv, cap = lib.ERR_INVALID_ARG, lib.ERR_CAPACITY
    n = 64
    assert forward(lib, dp, x_out=STEP * 1 + 16) == forward(lib, dp, h=STEP * 1) == forward(lib, dp, h=STEP * 2) == inv
    assert forward(lib, dp, h=STEP * 3) == forward(lib, dp, h=STEP * 6 + 2 * n) == forward(lib, dp, x_out=STEP * 2) == inv
    assert forward(lib, dp, x_out=STEP, s_x_out=2 * n) == inv  # the same place, another stride
    assert backward(lib, dp, dx=STEP * 2) == backward(lib, dp, dy=STEP * 4) == backward(lib, dp, dgate=STEP * 5) == cap
    for k, others in (("dx", (1, 3, 4, 5, 9, 10)), ("dy", (1, 2, 3, 5, 8, 10)), ("dgate", (1, 2, 3, 4, 8, 9))):
        for o in others:
            assert backward(lib, dp, **{k: STEP * o}) == inv, (k, o)
    assert backward(lib, dp, dx=STEP * 2, s_dx=2 * n) == inv
    # Columns of one wider tensor side by side do not meet.
    wide = dict(s_dx=3 * n, s_dy=3 * n, s_dgate=3 * n, dx=STEP * 20, dy=STEP * 20 + 2 * n, dgate=STEP * 20 + 4 * n)
    assert backward(lib, dp, **wide) == cap
    assert backward(lib, dp, **dict(wide, dgate=STEP * 20 + 4 * n - 16)) == inv
    assert backward(lib, dp, dw_pre=STEP * 11 + 4 * n - 4) == inv and backward(lib, dp, dw_pre=STEP * 11 + 4 * n) == cap


def test_binding_checks_on_host_tensors(lib, bound):
    p, dp = bound
    dplan = lib.DevicePlan(dp, p, None)
    x = torch.zeros(64, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        lib.residual_norm(x, x, None, dplan, -1, x, x)
    for bad in (x.half(), x[0], x[:5], None):
        with pytest.raises(ValueError, match="residual"):
            lib.residual_norm(bad, x, None, dplan, -1, x, x)
    with pytest.raises(ValueError, match="gate_fn"):
        lib.residual_norm(x, x, None, dplan, -1, x, x, gate_fn="tanh")


def test_widths_of_the_workloads(lib):
    for cfg in range(1, 6):
        w = synth.WORKLOADS[cfg]
        assert lib.residual_norm_ws_bytes(w.Hq * w.d) > 0


def test_outputs_on_weights_their_gradients_and_the_workspace(lib, bound):
    _, dp = bound
    inv, cap = lib.ERR_INVALID_ARG, lib.ERR_CAPACITY
    n, T = 64, 64
    row, ws = 2 * n, lib.residual_norm_ws_bytes(64)
    for k in ("x_out", "h"):
        for w in (4, 5):
            assert forward(lib, dp, **{k: STEP * w}) == inv, (k, w)
            assert forward(lib, dp, **{k: STEP * w + 4 * n - 16}) == inv, (k, w)
            assert forward(lib, dp, **{k: STEP * w - (T - 1) * row - 16}) == inv, (k, w)  # its last row
    for k in ("dx", "dy", "dgate"):
        for o, size in ((6, 4 * n), (7, 4 * n), (11, 4 * n), (12, 4 * n), (13, ws)):
            assert backward(lib, dp, **{k: STEP * o + size - 16}) == inv, (k, o)
            assert backward(lib, dp, **{k: STEP * o - (T - 1) * row - 16}) == inv, (k, o)
            assert backward(lib, dp, **{k: STEP * o + size}) == cap, (k, o)
            assert backward(lib, dp, **{k: STEP * o - T * row}) == cap, (k, o)
    for k, size in (("dw_post", 4 * n), ("dw_pre", 4 * n), ("ws", ws)):
        for o in (1, 2, 3, 4, 5):
            assert backward(lib, dp, **{k: STEP * o + T * row - 16}) == inv, (k, o)
            assert backward(lib, dp, **{k: STEP * o - size + 16}) == inv, (k, o)
            assert backward(lib, dp, **{k: STEP * o + T * row}) == backward(lib, dp, **{k: STEP * o - size}) == cap, (k, o)
        for o in (6, 7):
            assert backward(lib, dp, **{k: STEP * o}) == inv, (k, o)
    for k in ("dw_post", "dw_pre"):
        assert backward(lib, dp, **{k: STEP * 13 + ws - 4}) == inv and backward(lib, dp, **{k: STEP * 13 + ws}) == cap
    # Between the rows of a slice there is room; beside it too.
    for k, size in (("dw_post", 4 * n), ("dw_pre", 4 * n)):
        wide = dict(s_dx=4 * n, dx=STEP * 20)
        assert backward(lib, dp, **wide, **{k: STEP * 20 + 8 * n * 3 + row}) == cap, k
        assert backward(lib, dp, **wide, **{k: STEP * 20 + 8 * n * 3 + row - 4}) == inv, k
        assert backward(lib, dp, **wide, **{k: STEP * 20 + 8 * n * 4 - size + 4}) == inv, k
        assert backward(lib, dp, **wide, **{k: STEP * 20 + 8 * n * (T - 1) + row}) == cap, k


def test_session_backward_needs_a_residual(lib):
    from context_document_masked_gb300.session import CPAttention
    s = object.__new__(CPAttention)
    with pytest.raises(ValueError, match="x_out or dx_out"):
        s.residual_norm_backward(None, None, None)
