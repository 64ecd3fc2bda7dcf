"""Pins of the residual norm's oracle: torch autograd in fp64 and central differences."""
import itertools

import numpy as np
import pytest

from oracle import residual as R

torch = pytest.importorskip("torch")

FORMS = [(g, p, True) for g, p in itertools.product(["sigmoid", "plain", None], [True, False])] + [(None, True, False)]


@pytest.mark.parametrize("gate_fn,post_norm,block", FORMS)
def test_against_autograd_and_differences(gate_fn, post_norm, block):
    T, n, eps, a, b = 5, 12, 1e-3, 0.9, 0.3
    rng = np.random.default_rng(0)
    names = ["x"] + (["y", "w_post"] if block else []) + ["w_pre"] + (["z"] if gate_fn else [])
    v = {k: rng.normal(size=(n,) if k.startswith("w") else (T, n)) for k in names}
    dh, dX = rng.normal(size=(T, n)), rng.normal(size=(T, n))
    kw = dict(post_norm=post_norm, gate_fn=gate_fn or "plain", a=a, b=b, eps=eps)

    def loss(u):
        X, h = R.forward(u["x"], u.get("y"), u.get("z"), u.get("w_post"), u["w_pre"], **kw)
        return (X * dX).sum() + (h * dh).sum()

    t = {k: torch.tensor(x, requires_grad=True) for k, x in v.items()}
    X = a * t["x"]
    if block:
        u = t["y"] * (torch.rsqrt(t["y"].pow(2).mean(-1, keepdim=True) + eps) if post_norm else 1) * t["w_post"]
        if gate_fn:
            u = u * (torch.sigmoid(t["z"]) if gate_fn == "sigmoid" else t["z"])
        X = X + b * u
    h = X * torch.rsqrt(X.pow(2).mean(-1, keepdim=True) + eps) * t["w_pre"]
    grads = dict(zip(names, torch.autograd.grad((X * torch.tensor(dX)).sum() + (h * torch.tensor(dh)).sum(), list(t.values()))))
    fX, fh = R.forward(v["x"], v.get("y"), v.get("z"), v.get("w_post"), v["w_pre"], **kw)
    np.testing.assert_allclose(fX, X.detach().numpy(), atol=1e-13)
    np.testing.assert_allclose(fh, h.detach().numpy(), atol=1e-13)
    got = R.backward(dh, dX, fX, v.get("y"), v.get("z"), v.get("w_post"), v["w_pre"], **kw)
    for k in names:
        mine = got[{"z": "dgate"}.get(k, "d" + k)]
        np.testing.assert_allclose(mine, grads[k].numpy(), atol=1e-12)
        for at in ([(0,), (n - 1,)] if k.startswith("w") else [(0, 3), (T - 1, n - 1)]):
            ends = []
            for step in (1e-5, -1e-5):
                w = {q: y.copy() for q, y in v.items()}
                w[k][at] += step
                ends.append(loss(w))
            assert abs((ends[0] - ends[1]) / 2e-5 - mine[at]) < 1e-7


def test_parts_missing():
    x = np.arange(1.0, 9).reshape(1, 8)
    X, h = R.forward(x, eps=0)
    assert np.array_equal(X, x)
    np.testing.assert_allclose((h ** 2).mean(), 1)
    out = R.backward(None, x, x, y=x, post_norm=False, a=2.0, b=3.0)
    assert np.array_equal(out["dx"], 2 * x) and np.array_equal(out["dy"], 3 * x) and out["dw_pre"] is None
    np.testing.assert_allclose(R.gate(np.array([0.0, 800, -800, np.inf, -np.inf]), "sigmoid")[0], [0.5, 1, 0, 1, 0])
