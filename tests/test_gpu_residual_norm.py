"""The residual norm on the GPU and its gradient against the definition in 64 bits.

Bounds, element by element (u = 2^-24, fp32's half step; bf16's is 2^-8): a row's
sum runs over at most 8 to 16 values of a thread, 5 steps of a warp and 32 warps:
53u of the sum of its terms' sizes, every term with 2u of its own; a factor
1 / sqrt adds half of that and 4u: F = 32u. A gate's exponential has its argument
rounded (2u |z|) and 2^-21. The rest is counted operation by operation. A weight's
gradient adds T / 152 + 1 rows of a CTA at most, the CTAs in 32 runs and those."""
import numpy as np
import pytest
import torch

from oracle import residual as R

pytestmark = pytest.mark.gpu

U, BF16 = 2.0 ** -24, 2.0 ** -8
F = 32 * U


def session(docs, cp=1, policy="perdoc"):
    from context_document_masked_gb300.session import CPAttention
    return CPAttention(docs, cp, policy, 4, 2, 64)


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def make(T, n, seed=0, gate="sigmoid", block=True, res=torch.bfloat16, w=torch.float32, spread=1.0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, scale=1.0):
        return (scale * torch.randn(*shape, generator=g)).to(dtype).cuda()
    x = dict(x=normal(T, n, dtype=res, scale=spread), dx_out=normal(T, n, dtype=res), dh=normal(T, n))
    x["y"] = normal(T, n, scale=spread) if block else None
    x["gate"] = normal(T, n, scale=2) if block and gate else None
    x["w_post"] = (1 + 0.1 * normal(n, dtype=torch.float32)).to(w) if block and w else None
    x["w_pre"] = (1 + 0.1 * normal(n, dtype=torch.float32)).to(w) if w else None
    return x


def gate_error(z, fn):
    """Relative error of g(z), and of g'(z). (From |z| = 104 on exp(-|z|) is below 2^-150: g is 1 to the last bit or below
    every positive fp32 number, and the argument's rounding, 2u |z|, an infinite one's too, moves nothing any more.)"""
    if z is None or fn == "plain":
        return 0.0
    return 2 * U * np.minimum(np.abs(z), 104) + 2.0 ** -21 + 8 * U


def forward_reference(x, kw):
    v = {k: f64(t) for k, t in x.items()}
    a, b, fn, eps = kw["res_scale"], kw["branch_scale"], kw["gate_fn"], kw["eps"]
    X, h = R.forward(v["x"], v["y"], v["gate"], v["w_post"], v["w_pre"], kw["post_norm"], fn, a, b, eps)
    eX = 4 * U * (np.abs(a * v["x"]) + np.abs(X))
    if v["y"] is not None:
        eX = eX + np.abs(X - a * v["x"]) * (F + 6 * U + gate_error(v["gate"], fn))
    r = R.norm_factor(X, eps)
    w = 1.0 if v["w_pre"] is None else np.abs(v["w_pre"])
    er = (np.abs(X) * eX).mean(-1, keepdims=True) * r * r + F
    return dict(x_out=(X, eX), h=(h, np.abs(h) * (er + 4 * U) + eX * r * w))


def backward_reference(x, kw):
    v = {k: f64(t) for k, t in x.items()}
    a, b, fn, eps, post = kw["res_scale"], kw["branch_scale"], kw["gate_fn"], kw["eps"], kw["post_norm"]
    X, T = v["x"], len(v["x"])
    want = R.backward(v["dh"], v["dx_out"], X, v["y"], v["gate"], v["w_post"], v["w_pre"], post, fn, a, b, eps)
    D = want["dx"] / a
    eD = 4 * U * (np.abs(D) + (0 if v["dx_out"] is None else np.abs(v["dx_out"])))
    chain = (T / 152 + 1 + 40 + 32) * U
    err = {}
    if v["dh"] is not None:
        r = R.norm_factor(X, eps)
        k = v["dh"] * (1.0 if v["w_pre"] is None else v["w_pre"])
        mean, size = np.mean(k * X, -1, keepdims=True), np.mean(np.abs(k * X), -1, keepdims=True)
        eD = eD + np.abs(r * k) * (F + 4 * U) + np.abs(X) * r ** 3 * (64 * U * size + (3 * F + 8 * U) * np.abs(mean))
        terms = np.abs(v["dh"] * X * r).sum(0)
        err["dw_pre"] = terms * (F + 4 * U + chain)
    err["dx"] = abs(a) * eD + 2 * U * np.abs(want["dx"])
    if v["y"] is not None:
        y, w = v["y"], 1.0 if v["w_post"] is None else v["w_post"]
        ry, Fy = (R.norm_factor(y, eps), F) if post else (1.0, 0.0)
        g, dg = R.gate(v["gate"], fn)
        eg = gate_error(v["gate"], fn)
        if v["gate"] is not None:
            err["dgate"] = np.abs(b * (y * ry * w) * dg) * eD + np.abs(want["dgate"]) * (Fy + 8 * U + 2 * eg)
        c, ec = b * D * g, abs(b) * np.abs(g) * (eD + np.abs(D) * (4 * U + eg))
        err["dw_post"] = (np.abs(y * ry) * (ec + np.abs(c) * (Fy + 4 * U + chain))).sum(0)
        e, ee = c * w, ec * np.abs(w) + 2 * U * np.abs(c * w)
        err["dy"] = ry * ee + np.abs(ry * e) * (Fy + 4 * U)
        if post:
            mean, size = np.mean(e * y, -1, keepdims=True), np.mean(np.abs(e * y), -1, keepdims=True)
            emean = 64 * U * size + np.mean(ee * np.abs(y), -1, keepdims=True)
            err["dy"] = err["dy"] + np.abs(y) * ry ** 3 * (emean + (3 * F + 8 * U) * np.abs(mean))
    return {k: (want[k], err[k]) for k in err}


def within(got, want, name):
    ref, err = want
    half = BF16 if got.dtype == torch.bfloat16 else U
    over = np.abs(f64(got) - ref) - (1 + half) * err - half * np.abs(ref)
    assert (over <= 1e-37).all(), f"{name}: {float(over.max())} over its bound"


KW = dict(post_norm=True, gate_fn="sigmoid", res_scale=0.96, branch_scale=0.28, eps=1e-6)


def run_forward(s, x, kw, **more):
    return s.residual_norm(x["x"], x["y"], x["gate"], w_post=x["w_post"], w_pre=x["w_pre"], **kw, **more)


def run_backward(s, x, kw, **more):
    out = s.residual_norm_backward(x["dh"], x["dx_out"], x["x"], x["y"], x["gate"], w_post=x["w_post"], w_pre=x["w_pre"],
                                   **kw, **more)
    return dict(zip(("dx", "dy", "dgate", "dw_post", "dw_pre"), out))


def check(s, x, kw):
    want = forward_reference(x, kw)
    for name, y in zip(("x_out", "h"), run_forward(s, x, kw)):
        within(y, want[name], name)
    got, want = run_backward(s, x, kw), backward_reference(x, kw)
    for name, y in got.items():
        if y is not None:
            within(y, want[name], name)
    return got


@pytest.mark.parametrize("T,n", [(1, 8), (5, 64), (130, 256), (301, 768), (64, 1000), (9, 2048), (9, 2056), (200, 4096),
                                 (33, 8192), (5, 16384), (7, 16376), (2000, 72)])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_sizes(cuda, T, n, res):
    check(session([T]), make(T, n, seed=n, res=res), KW)


@pytest.mark.parametrize("gate", ["sigmoid", "plain", None])
@pytest.mark.parametrize("post_norm", [True, False])
@pytest.mark.parametrize("w", [torch.bfloat16, torch.float32, None])
def test_forms(cuda, gate, post_norm, w):
    x = make(77, 264, gate=gate, w=w)
    got = check(session([50, 27]), x, dict(KW, post_norm=post_norm, gate_fn=gate or "plain"))
    assert (got["dgate"] is None) == (gate is None) and (got["dw_pre"] is None) == (w is None)


def test_no_block_and_no_norm(cuda):
    s = session([40])
    x = make(40, 128, block=False)
    kw = dict(KW, res_scale=1.0)
    x_out, h = run_forward(s, x, kw)
    assert x_out is x["x"]
    within(h, forward_reference(x, kw)["h"], "h")
    got, want = run_backward(s, x, kw), backward_reference(x, kw)
    assert got["dy"] is None and got["dgate"] is None and got["dw_post"] is None
    within(got["dx"], want["dx"], "dx")
    within(got["dw_pre"], want["dw_pre"], "dw_pre")
    # The first gradient of a stack has nothing along the residual, the last block no norm behind it.
    x = dict(make(40, 128), dx_out=None)
    for name, y in run_backward(s, x, KW).items():
        within(y, backward_reference(x, KW)[name], name)
    x = dict(make(40, 128), dh=None, w_pre=None)
    x_out, h = run_forward(s, x, KW, pre_norm=False)
    assert h is None
    within(x_out, forward_reference(x, KW)["x_out"], "x_out")
    got = run_backward(s, x, KW)
    assert got["dw_pre"] is None
    for name in ("dx", "dy", "dgate", "dw_post"):
        within(got[name], backward_reference(x, KW)[name], name)


@pytest.mark.parametrize("policy,cp", [("perdoc", 3), ("wholedoc", 2)])
def test_shards(cuda, policy, cp):
    """One shard after another: only its rows are written, the weights' gradients add up."""
    docs = [1, 130, 300, 2, 77, 2]
    s, n = session(docs, cp, policy), 136
    T = sum(docs)
    x = make(T, n, seed=4)
    fwd, bwd = forward_reference(x, KW), backward_reference(x, KW)
    nan = torch.full((T, n), torch.nan, dtype=torch.bfloat16, device="cuda")
    outs = {k: nan.clone() for k in ("x_out", "h")}
    grads = {k: nan.clone() for k in ("dx", "dy", "dgate")}
    dw = {k: torch.zeros(n, device="cuda") for k in ("dw_post", "dw_pre")}
    done = torch.zeros(T, dtype=torch.bool, device="cuda")
    for j in range(cp):
        run_forward(s, x, KW, shard=j, **outs)
        run_backward(s, x, KW, shard=j, **grads, **dw)
        done[torch.from_numpy(s.plan.query_indices(j)).cuda().long()] = True
        for y in (*outs.values(), *grads.values()):
            assert torch.equal(y.isnan().any(1), ~done) and torch.equal(y.isnan().all(1), ~done)
    for k, y in outs.items():
        within(y, fwd[k], k)
    for k, y in (grads | dw).items():
        within(y, bwd[k], k)


def test_many_short_documents(cuda):
    """Shards of many runs of a few rows, which are taken run by run."""
    docs = [1, 2, 5] * 600
    s, n = session(docs, 2, "wholedoc"), 64
    T = sum(docs)
    x = make(T, n, seed=4)
    fwd, bwd = forward_reference(x, KW), backward_reference(x, KW)
    outs = {k: torch.full((T, n), torch.nan, dtype=torch.bfloat16, device="cuda") for k in ("x_out", "h", "dx", "dy", "dgate")}
    dw = {k: torch.zeros(n, device="cuda") for k in ("dw_post", "dw_pre")}
    for j in range(2):
        run_forward(s, x, KW, shard=j, x_out=outs["x_out"], h=outs["h"])
        run_backward(s, x, KW, shard=j, dx=outs["dx"], dy=outs["dy"], dgate=outs["dgate"], **dw)
    for k, y in (outs | dw).items():
        within(y, (fwd | bwd)[k], k)


def test_a_shard_without_tokens(cuda):
    s = session([3], 4, "perdoc")
    empty = [j for j in range(4) if len(s.plan.query_indices(j)) == 0]
    assert empty
    x = make(3, 64)
    out = run_backward(s, x, KW, shard=empty[0], dw_post=torch.ones(64, device="cuda"), dw_pre=torch.ones(64, device="cuda"),
                       zero_grads=True)
    assert out["dw_post"].abs().max() == 0 and out["dw_pre"].abs().max() == 0
    run_forward(s, x, KW, shard=empty[0])


def test_slices_and_in_place(cuda):
    """Operands inside wider tensors, the residual and the gradients in place; neighbours stay as they were."""
    T, n = 100, 96
    s = session([T])
    x = make(T, n, seed=8)
    fwd, bwd = forward_reference(x, KW), backward_reference(x, KW)
    wide = torch.zeros(T, 3 * n, dtype=torch.bfloat16, device="cuda")
    y, gate, h = wide[:, :n], wide[:, n:2 * n], wide[:, 2 * n:]
    y.copy_(x["y"]), gate.copy_(x["gate"])
    residual = x["x"].clone()
    s.residual_norm(residual, y, gate, w_post=x["w_post"], w_pre=x["w_pre"], x_out=residual, h=h, **KW)
    within(residual, fwd["x_out"], "x_out")
    within(h, fwd["h"], "h")
    assert torch.equal(y, x["y"]) and torch.equal(gate, x["gate"])
    dx = x["dx_out"].clone()
    s.residual_norm_backward(x["dh"], dx, x["x"], y, gate, w_post=x["w_post"], w_pre=x["w_pre"], dx=dx, dy=y, dgate=gate, **KW)
    for name, t in (("dx", dx), ("dy", y), ("dgate", gate)):
        within(t, bwd[name], name)
    within(h, fwd["h"], "h")


def test_weights_gradients_are_added_and_repeat(cuda):
    T, n = 5000, 256
    s = session([T])
    x = make(T, n, seed=2)
    a, b = run_backward(s, x, KW), run_backward(s, x, KW)
    assert all(torch.equal(a[k], b[k]) for k in a)  # a fixed order
    start = torch.arange(n, dtype=torch.float32, device="cuda")
    c = run_backward(s, x, KW, dw_post=start.clone())
    torch.testing.assert_close(c["dw_post"], a["dw_post"] + start, rtol=2 * U, atol=0)
    assert torch.equal(c["dw_pre"], a["dw_pre"])
    d = run_backward(s, x, KW, dw_post=torch.full((n,), torch.nan, device="cuda"), zero_grads=True)
    assert torch.equal(d["dw_post"], a["dw_post"])


@pytest.mark.parametrize("spread", [1e-18, 1e-3, 300.0, 1e17])
def test_sizes_of_values(cuda, spread):
    """Sums of squares up to 1e34 * n; rows far below eps."""
    check(session([30]), make(30, 512, seed=6, spread=spread), KW)


def test_odd_values(cuda):
    """Rows of zeros, gates at the ends of the sigmoid and infinite, a NaN that stays in its row."""
    T, n = 6, 256
    x = make(T, n, seed=5)
    x["y"][0] = 0
    x["x"][1] = 0
    x["y"][1] = 0
    x["gate"][2, :4] = torch.tensor([90.0, -90.0, 3e38, -3e38], device="cuda")
    x["gate"][3, :2] = torch.tensor([torch.inf, -torch.inf], device="cuda")
    check(session([T]), x, KW)
    s = session([T])
    x["x"][4, 7] = torch.nan
    x_out, h = run_forward(s, x, KW)
    got = run_backward(s, x, KW)
    rest = torch.tensor([0, 1, 2, 3, 5], device="cuda")
    assert h[4].isnan().all() and not h[rest].isnan().any() and not x_out[rest].isnan().any()
    for k in ("dx", "dy", "dgate"):
        assert got[k][4].isnan().any() and not got[k][rest].isnan().any()


def test_streams_and_graphs(cuda):
    """A captured forward and backward, replayed with new inputs beside eager calls on another stream."""
    T, n = 700, 768
    s = session([T])
    x1, x2 = make(T, n, seed=1), make(T, n, seed=2)
    bufs = {k: t.clone() for k, t in x1.items()}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run_forward(s, bufs, KW), run_backward(s, bufs, KW)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        fwd, bwd = run_forward(s, bufs, KW), run_backward(s, bufs, KW)
    for k, t in bufs.items():
        t.copy_(x2[k])
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph.replay()
    eager = run_backward(s, x1, KW)
    other = run_backward(s, x2, KW, stream=torch.cuda.Stream().cuda_stream)
    torch.cuda.synchronize()
    for got, x in ((bwd, x2), (eager, x1), (other, x2)):
        want = backward_reference(x, KW)
        for k, y in got.items():
            within(y, want[k], k)
    want = forward_reference(x2, KW)
    within(fwd[0], want["x_out"], "x_out")
    within(fwd[1], want["h"], "h")


def test_binding_refusals(cuda):
    s = session([20])
    x = make(20, 64)
    for bad in (dict(y=x["y"].float()), dict(y=x["y"][:10]), dict(gate=x["gate"].t().contiguous().t()),
                dict(y=x["y"][:, ::2].contiguous()), dict(w_pre=x["w_pre"].double()), dict(w_pre=x["w_pre"][:32]),
                dict(w_post=x["w_post"].bfloat16()), dict(x=x["x"].half())):
        with pytest.raises(ValueError):
            run_forward(s, dict(x, **bad), KW)
    with pytest.raises(ValueError):
        run_backward(s, dict(x, dx_out=x["dx_out"].float()), KW)
    from context_document_masked_gb300 import fcp
    with pytest.raises(fcp.FcpError):
        run_forward(s, x, KW, h=x["y"])


# Rows of more than 8192 values: the forward's ring where it fits the shared memory, the gradient by pairs of CTAs. (A pair adds
# T / 76 + 1 rows of a weight's gradient, and a warp of the last sum 3 of theirs, not 40: for T <= 5624 within the bound above.)
@pytest.mark.parametrize("T,n", [(1, 8200), (200, 8208), (311, 9216), (90, 11464), (77, 12296), (160, 16384)])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_wide_rows(cuda, T, n, res):
    check(session([T]), make(T, n, seed=n, res=res), KW)


@pytest.mark.parametrize("gate,post_norm,w", [("plain", True, torch.bfloat16), (None, False, torch.float32), (None, True, None),
                                              ("sigmoid", False, torch.float32)])
def test_wide_forms(cuda, gate, post_norm, w):
    x = make(170, 10008, gate=gate, w=w)
    check(session([100, 70]), x, dict(KW, post_norm=post_norm, gate_fn=gate or "plain"))


def test_wide_rows_without_a_block_of_shards_repeat(cuda):
    docs = [1, 2, 5] * 210  # so many runs that they are taken whole
    s, n, T = session(docs, 1, "wholedoc"), 8712, 8 * 210
    x, kw = make(T, n, seed=3), dict(KW)
    fwd, bwd = forward_reference(x, kw), backward_reference(x, kw)
    first = run_backward(s, x, kw, shard=0)
    again = run_backward(s, x, kw, shard=0)
    for k, y in first.items():
        assert torch.equal(y, again[k])
        within(y, bwd[k], k)
    for k, y in zip(("x_out", "h"), run_forward(s, x, kw, shard=0)):
        within(y, fwd[k], k)
    x = make(90, n, block=False, res=torch.float32)
    kw = dict(KW, res_scale=1.0)
    got, want = run_backward(session([90]), x, kw), backward_reference(x, kw)
    within(got["dx"], want["dx"], "dx")
    within(got["dw_pre"], want["dw_pre"], "dw_pre")


def test_rows_past_32_bits(cuda):
    """Columns of one tensor of 2.6 G values (5.2 GB): the same results as from tensors of their own, whose first and last
    rows are the definition's."""
    T, n, width = 40000, 64, 65536
    s = session([15000, 25000], 2)
    x = make(T, n, seed=11)
    wide = torch.empty(T, width, dtype=torch.bfloat16, device="cuda")

    def column(i, t=None):
        c = wide[:, width - (i + 1) * n:width - i * n]
        return c.fill_(-7) if t is None else c.copy_(t)
    far = {k: column(i, x[k]) for i, k in enumerate(("x", "y", "gate", "dx_out", "dh"))}
    far = dict(x, **far)
    names = ("x_out", "h", "dx", "dy", "dgate")
    outs = {k: column(5 + i) for i, k in enumerate(names)}
    run_forward(s, far, KW, x_out=outs["x_out"], h=outs["h"])
    dw = run_backward(s, far, KW, dx=outs["dx"], dy=outs["dy"], dgate=outs["dgate"])
    near = dict(zip(names, run_forward(s, x, KW))) | run_backward(s, x, KW)
    for k in names:
        assert torch.equal(outs[k], near[k]), k
    for k in ("dw_post", "dw_pre"):
        assert torch.equal(dw[k], near[k])
    for rows in (slice(0, 40), slice(T - 40, T)):
        part = {k: t[rows] if t is not None and t.dim() == 2 else t for k, t in x.items()}
        want = forward_reference(part, KW) | {k: v for k, v in backward_reference(part, KW).items() if not k.startswith("dw")}
        for k in names:
            within(near[k][rows], want[k], k)


@pytest.mark.parametrize("T,n", [(130, 256), (77, 1000), (9, 2056), (200, 4096), (33, 8192), (90, 9216)])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_bf16_weights(cuda, T, n, res):
    check(session([T]), make(T, n, seed=n, res=res, w=torch.bfloat16), KW)
