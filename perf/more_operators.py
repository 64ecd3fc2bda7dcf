"""Workloads of a sliding-window layer: windowed attention and the norms around its blocks.

Two operators, each with its gradient, over a packed sequence:

  window_attn         document-masked attention in which a token sees the last `window`
                      tokens of its document, itself among them, and the document's first
                      `sinks` tokens.
  window_attn_step    the same forward and the gradients of Q, K and V.
  residual_norm       the stream between two blocks: a block's output normed, gated, scaled and
                      added to the residual, and the norm before the next block.
  residual_norm_grad  its gradient, that of both norms' weights among it.

`run` computes them in elementary torch operations, or with `own` through this
package's session.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------- cases


def listed():
    return [
        # Short documents of a small model, little more than a window each: a call that is all latency.
        dict(name="window_attn 2k h4 d64 w128", op="window_attn", T=2048, hq=4, hkv=2, d=64, window=128, sinks=4,
             docs="uniform 64 640", doc_seed=1, cp=2, policy="llama3"),
        # Odd length and window, groups of three heads, one sink.
        dict(name="window_attn 5003 h6 w300", op="window_attn", T=5003, hq=6, hkv=2, d=128, window=300, sinks=1,
             docs="lognormal 6.5 1.2 1 4096", doc_seed=5, cp=1, policy="perdoc"),
        # The 32K packed sequence of a 32/8-head layer.
        dict(name="window_attn 32k h32 w1024", op="window_attn", T=32768, hq=32, hkv=8, d=128, window=1024, sinks=4,
             docs="lognormal 7.5 1.2 32 32768", doc_seed=1002, cp=4, policy="perdoc"),
        # One long document over sixteen shards, the widest usual window: the forward's largest.
        dict(name="window_attn 64k h32 w4096", op="window_attn", T=65536, hq=32, hkv=8, d=128, window=4096, sinks=4,
             docs="one", doc_seed=6, cp=16, policy="perdoc"),
        # Training steps: as many KV as query heads, no sinks ...
        dict(name="window_attn_step 4k h12 d64 w256", op="window_attn_step", T=4096, hq=12, hkv=12, d=64, window=256,
             sinks=0, docs="uniform 64 640", doc_seed=3, cp=2, policy="perdoc"),
        # ... an odd length and a window shorter than a tile ...
        dict(name="window_attn_step 7001 h6 w100", op="window_attn_step", T=7001, hq=6, hkv=2, d=128, window=100,
             sinks=4, docs="lognormal 6.5 1.2 1 4096", doc_seed=5, cp=1, policy="perdoc"),
        # ... the 32K packed sequence with a short window ...
        dict(name="window_attn_step 32k h32 w128", op="window_attn_step", T=32768, hq=32, hkv=8, d=128, window=128,
             sinks=4, docs="lognormal 7.5 1.2 32 32768", doc_seed=1002, cp=4, policy="perdoc"),
        # ... and one long document over eight shards: the largest.
        dict(name="window_attn_step 64k h16 w2048", op="window_attn_step", T=65536, hq=16, hkv=2, d=128, window=2048,
             sinks=16, docs="one", doc_seed=6, cp=8, policy="perdoc"),
        # Norms: a small model's rows (latency) ...
        dict(name="residual_norm 2k n256", op="residual_norm", T=2048, n=256, gate="none", post_norm=True,
             residual="bf16", hq=4, hkv=2, d=64, docs="uniform 64 640", doc_seed=1, cp=2, policy="llama3"),
        # ... and 64K tokens of the widest layer, gated.
        dict(name="residual_norm 64k n8192", op="residual_norm", T=65536, n=8192, gate="sigmoid", post_norm=True,
             residual="bf16", hq=64, hkv=8, d=128, docs="mix 128 1024 4096 16384", doc_seed=4, cp=16,
             policy="wholedoc"),
        # Gradients: a ragged batch with an fp32 residual ...
        dict(name="residual_norm_grad 5003 n768", op="residual_norm_grad", T=5003, n=768, gate="sigmoid",
             post_norm=False, residual="fp32", hq=12, hkv=12, d=64, docs="lognormal 5.0 1.2 1 2048", doc_seed=2, cp=1,
             policy="perdoc"),
        # ... and the 32K packed sequence of a 32-head layer.
        dict(name="residual_norm_grad 32k n4096", op="residual_norm_grad", T=32768, n=4096, gate="sigmoid",
             post_norm=True, residual="bf16", hq=32, hkv=8, d=128, docs="lognormal 7.5 1.2 32 32768", doc_seed=1002,
             cp=4, policy="perdoc"),
    ]


HEADS = [(4, 2, 64), (5, 5, 64), (8, 1, 64), (12, 12, 64), (6, 2, 128), (16, 2, 128), (32, 8, 128), (64, 8, 128)]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window_attn", "window_attn_step", "residual_norm", "residual_norm_grad"])
    hq, hkv, d = rng.choice(HEADS)
    low = 64 if op == "window_attn_step" else 1  # a document of one token has no gradient of Q and K
    c = dict(op=op, T=_log_uniform(rng, low, 65536), hq=hq, hkv=hkv, d=d,
             docs=rng.choice(["one", "uniform 64 640", "uniform 1 200", "lognormal 5.0 1.2 1 2048",
                              "lognormal 7.5 1.2 32 32768", "mix 128 1024 4096 16384"]),
             doc_seed=rng.randrange(1 << 20), cp=rng.choice([1, 2, 4, 8]), policy="perdoc")
    if op.startswith("window"):
        # A window of one token leaves Q and K without a gradient.
        c.update(window=_log_uniform(rng, 8 if op == "window_attn_step" else 1, 8192),
                 sinks=rng.choice([0, 0, 1, 4, 4, 16, 37, 64]))
    else:
        c.update(n=8 * _log_uniform(rng, 8, 1024), gate=rng.choice(["none", "sigmoid", "plain"]),
                 post_norm=rng.random() < 0.7, residual=rng.choice(["bf16", "fp32"]))
    most = [work(x) for x in listed() if x["op"] == op]
    most = {k: max(m[k] for m in most) for k in ("bytes", "flops")}
    while work(c)["flops"] > most["flops"] or work(c)["bytes"] > most["bytes"]:
        c["T"] = max(1, c["T"] * 2 // 3)
    return c


def doc_lengths(case):
    """Document lengths drawn one after another, the last one cut to fill T tokens."""
    kind, *a = case["docs"].split()
    a = [float(x) for x in a]
    rng = np.random.default_rng(case["doc_seed"])
    if kind == "one":
        return [case["T"]]
    out, total = [], 0
    while total < case["T"]:
        if kind == "uniform":
            n = rng.integers(int(a[0]), int(a[1]) + 1)
        elif kind == "lognormal":
            n = np.clip(np.rint(rng.lognormal(a[0], a[1])), a[2], a[3])
        else:  # one document in ten from the second range
            n = rng.integers(int(a[2]), int(a[3]) + 1) if rng.random() < 0.1 else rng.integers(int(a[0]), int(a[1]) + 1)
        n = min(int(n), case["T"] - total)
        out.append(n)
        total += n
    return out


def visible_pairs(case):
    """Pairs of a query and a key that it sees."""
    w, s, pairs = case["window"], case["sinks"], 0
    for n in doc_lengths(case):
        at = np.arange(n, dtype=np.int64)
        pairs += int(np.minimum(at + 1, w).sum() + np.clip(at - w + 1, 0, s).sum())
    return pairs


def work(case):
    T = case["T"]
    if case["op"].startswith("residual_norm"):
        n, res = case["n"], 4 if case["residual"] == "fp32" else 2
        gated = case["gate"] != "none"
        if case["op"] == "residual_norm":  # residual in and out, the block's output (and gate) in, the normed rows out
            return {"bytes": T * n * (2 * res + 2 + 2 * gated + 2) + 8 * n, "flops": 14 * T * n}
        # The residual and its gradient, the block's output (and gate), the gradient of the normed rows in; the
        # gradients of the residual, the block's output (and gate) and the weights out.
        return {"bytes": T * n * (3 * res + 2 + 2 + 2 + 4 * gated) + 16 * n, "flops": 36 * T * n}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    pairs = visible_pairs(case)
    if case["op"] == "window_attn":
        return {"bytes": T * (2 * hq + 2 * hkv) * d * 2 + hq * T * 4, "flops": 4 * d * hq * pairs}
    return {"bytes": T * (4 * hq + 4 * hkv) * d * 2 + hq * T * 4, "flops": 14 * d * hq * pairs}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    T = case["T"]
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    lengths = doc_lengths(case)
    s = dict(case=case, lengths=lengths, session=None)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    window = {}
    if case["op"].startswith("window"):
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        s["q"], s["k"], s["v"] = normal(T, hq, d), normal(T, hkv, d), normal(T, hkv, d)
        if case["op"] == "window_attn_step":
            s["do"] = normal(T, hq, d)
        window = dict(window=case["window"], sinks=case["sinks"])
    else:
        n = case["n"]
        res = torch.float32 if case["residual"] == "fp32" else torch.bfloat16
        s["x"] = normal(T, n, dtype=res)  # the residual: before the block, or (gradient) after it
        s["y"] = normal(T, n)             # the block's output
        s["gate"] = None if case["gate"] == "none" else normal(T, n)
        s["w_post"] = 1 + 0.1 * normal(n, dtype=torch.float32)
        s["w_pre"] = 1 + 0.1 * normal(n, dtype=torch.float32)
        # Residual scales of a deep stack.
        s["options"] = dict(post_norm=case["post_norm"], res_scale=0.96, branch_scale=0.28, eps=EPS)
        if case["gate"] != "none":
            s["options"]["gate_fn"] = case["gate"]
        if case["op"] == "residual_norm_grad":
            s["dh"] = normal(T, n)
            s["dx"] = normal(T, n, dtype=res)
    if own:
        from context_document_masked_gb300.session import CPAttention

        s["session"] = CPAttention(lengths, case["cp"], case["policy"], case["hq"], case["hkv"], case["d"], device=dev,
                                   **window)
    return s


# --------------------------------------------------------------- operators


def run(s):
    op = s["case"]["op"]
    if op == "residual_norm":
        return own_residual_norm(s) if own else plain_residual_norm(s)
    if op == "residual_norm_grad":
        return own_residual_norm_grad(s) if own else plain_residual_norm_grad(s)
    return own_window_attn(s) if own else plain_window_attn(s)


def own_window_attn(s):
    a, q, k, v = s["session"], s["q"], s["k"], s["v"]
    a.gather(k, v)
    if s["case"]["op"] == "window_attn":
        out, lse = a.forward(q, k, v)
        return {"out": out, "lse": lse}
    out, lse = a.forward(q, k, v, out_dtype=torch.float32)
    grads = a.backward(q, k, v, out, lse, s["do"])
    # The next layers take bf16, the type of the tensors that these are the gradients of.
    return dict(zip(("out", "dq", "dk", "dv"), (x.to(torch.bfloat16) for x in (out, *grads))), lse=lse)


def own_residual_norm(s):
    x, h = s["session"].residual_norm(s["x"], s["y"], s["gate"], w_post=s["w_post"], w_pre=s["w_pre"], **s["options"])
    return {"x": x, "h": h}


def own_residual_norm_grad(s):
    dx, dy, dgate, dw_post, dw_pre = s["session"].residual_norm_backward(
        s["dh"], s["dx"], s["x"], s["y"], s["gate"], w_post=s["w_post"], w_pre=s["w_pre"], **s["options"])
    out = {"dx": dx, "dy": dy, "dw_post": dw_post, "dw_pre": dw_pre}
    return out if dgate is None else dict(out, dgate=dgate)


def key_ranges(begin, a, b, window, sinks):
    """The keys that queries a .. b - 1 of a document that begins at `begin` may see, as one or two ranges."""
    first = max(begin, a - window + 1)
    last_sink = min(begin + sinks, b)
    return [(begin, b)] if first <= last_sink else [r for r in ((begin, last_sink), (first, b)) if r[0] < r[1]]


def plain_window_attn(s):
    case = s["case"]
    T, hq, hkv, d, G = case["T"], case["hq"], case["hkv"], case["d"], case["hq"] // case["hkv"]
    window, sinks, scale = case["window"], case["sinks"], 1 / math.sqrt(case["d"])
    grad = case["op"] == "window_attn_step"
    q, k, v = (s[x].float().transpose(0, 1) for x in "qkv")
    do = s["do"].float().transpose(0, 1) if grad else None
    out, lse = torch.empty_like(q), q.new_empty(hq, T)
    dq, dk, dv = (torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)) if grad else (None, None, None)
    begin = 0
    for n in s["lengths"]:  # nothing passes between documents
        for a in range(begin, begin + n, 1024):  # and a block of queries needs its window's keys and the sinks
            b = min(a + 1024, begin + n)
            ranges = key_ranges(begin, a, b, window, sinks)
            key = torch.cat([torch.arange(x, y, device="cuda") for x, y in ranges])
            kb = torch.cat([k[:, x:y] for x, y in ranges], 1)
            vb = torch.cat([v[:, x:y] for x, y in ranges], 1)
            distance = torch.arange(a, b, device="cuda")[:, None] - key
            hidden = (distance < 0) | ((distance >= window) & (key >= begin + sinks))
            qb = q[:, a:b].reshape(hkv, G * (b - a), d)
            p = (qb @ kb.transpose(1, 2)).mul_(scale).view(hkv, G, b - a, -1).masked_fill_(hidden, -math.inf)
            m = p.amax(-1, keepdim=True)
            p = p.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            p = p.div_(l).view(hkv, G * (b - a), -1)
            o = p @ vb
            out[:, a:b] = o.view(hq, b - a, d)
            lse[:, a:b] = (m + l.log()).view(hq, b - a)
            if grad:
                dob = do[:, a:b].reshape(hkv, G * (b - a), d)
                ds = (dob @ vb.transpose(1, 2)).sub_((dob * o).sum(-1, keepdim=True)).mul_(p)
                dq[:, a:b] = (ds @ kb).mul_(scale).view(hq, b - a, d)
                dkb, dvb = (ds.transpose(1, 2) @ qb).mul_(scale), p.transpose(1, 2) @ dob
                at = 0
                for x, y in ranges:
                    dk[:, x:y] += dkb[:, at:at + y - x]
                    dv[:, x:y] += dvb[:, at:at + y - x]
                    at += y - x
        begin += n
    if not grad:
        return {"out": out.transpose(0, 1).to(torch.bfloat16), "lse": lse}
    out, dq, dk, dv = (x.transpose(0, 1).to(torch.bfloat16) for x in (out, dq, dk, dv))
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def branch(s):
    """A block's output in 32 bits, normed where it is, with its weights; the gate's values; the norm's factor."""
    y = s["y"].float()
    r = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) if s["case"]["post_norm"] else 1.0
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    if s["case"]["gate"] == "sigmoid":
        gate = 1 / (1 + (-gate).exp())
    return y * r, gate, r


def plain_residual_norm(s):
    o = s["options"]
    y, gate, _ = branch(s)
    x = o["res_scale"] * s["x"].float() + o["branch_scale"] * gate * (y * s["w_post"])
    h = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["w_pre"]
    return {"x": x.to(s["x"].dtype), "h": h.to(torch.bfloat16)}


def plain_residual_norm_grad(s):
    o = s["options"]
    x, dh = s["x"].float(), s["dh"].float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xn = x * r
    g = dh * s["w_pre"]
    dx = s["dx"].float() + r * (g - xn * (g * xn).mean(-1, keepdim=True))
    yn, gate, ry = branch(s)
    du = o["branch_scale"] * dx
    out = {"dx": (o["res_scale"] * dx).to(s["x"].dtype), "dw_pre": (dh * xn).sum(0)}
    if s["gate"] is not None:
        dgate = du * (yn * s["w_post"])
        if s["case"]["gate"] == "sigmoid":
            dgate = dgate * gate * (1 - gate)
        out["dgate"] = dgate.to(torch.bfloat16)
    du = du * gate
    out["dw_post"] = (du * yn).sum(0)
    gy = du * s["w_post"]
    dy = ry * (gy - yn * (gy * yn).mean(-1, keepdim=True)) if s["case"]["post_norm"] else gy
    out["dy"] = dy.to(torch.bfloat16)
    return out


# ------------------------------------------------------- 64-bit definitions


def exact(case, seed):
    if case["op"].startswith("residual_norm"):
        return exact_residual_norm(prepare(case, seed))
    if work(case)["flops"] > 1e13:  # over what the 64-bit units do in the time there is
        return None
    return exact_window_attn(prepare(case, seed))


def exact_window_attn(s):
    """Head by head, blocks of 512 queries against their document's keys that the mask leaves; gradients by
    automatic differentiation."""
    case = s["case"]
    T, hq, hkv, d = case["T"], case["hq"], case["hkv"], case["d"]
    G, grad = hq // hkv, case["op"] == "window_attn_step"
    new = dict(dtype=torch.float64, device="cuda")
    out, lse, dq = torch.zeros(T, hq, d, **new), torch.zeros(hq, T, **new), torch.zeros(T, hq, d, **new)
    dk, dv = torch.zeros(T, hkv, d, **new), torch.zeros(T, hkv, d, **new)
    at = 0
    for n in s["lengths"]:
        for a in range(at, at + n, 512):
            b = min(a + 512, at + n)
            i = torch.arange(a, b, device="cuda")[:, None]
            j = torch.arange(at, b, device="cuda")
            j = j[(j - at < case["sinks"]) | (a - j < case["window"])]
            seen = (j <= i) & ((i - j < case["window"]) | (j - at < case["sinks"]))
            for g in range(hkv):
                k, v = (s[x][j, g].double().requires_grad_(grad) for x in "kv")
                q = s["q"][a:b, g * G:(g + 1) * G].double().transpose(0, 1).contiguous().requires_grad_(grad)
                score = torch.where(seen, q @ k.T / math.sqrt(d), -math.inf)
                o = torch.softmax(score, -1) @ v
                out[a:b, g * G:(g + 1) * G] = o.detach().transpose(0, 1)
                lse[g * G:(g + 1) * G, a:b] = torch.logsumexp(score.detach(), -1)
                if grad:
                    do = s["do"][a:b, g * G:(g + 1) * G].double().transpose(0, 1)
                    gq, gk, gv = torch.autograd.grad(o, (q, k, v), do)
                    dq[a:b, g * G:(g + 1) * G] = gq.transpose(0, 1)
                    dk[:, g].index_add_(0, j, gk)
                    dv[:, g].index_add_(0, j, gv)
        at += n
    if not grad:
        return {"out": out, "lse": lse}
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def exact_residual_norm(s):
    """From the definition, blocks of rows at a time; gradients by automatic differentiation."""
    case, o = s["case"], s["options"]
    grad = case["op"] == "residual_norm_grad"
    w_post, w_pre = (s[x].double().requires_grad_(grad) for x in ("w_post", "w_pre"))
    blocks, weights = [], [0, 0]
    for a in range(0, case["T"], 4096):
        rows = slice(a, min(a + 4096, case["T"]))
        x, y = (s[name][rows].double().requires_grad_(grad) for name in ("x", "y"))
        leaves = [y, w_post]
        u = y * w_post
        if case["post_norm"]:
            u = u / (y.pow(2).sum(-1, keepdim=True) / case["n"] + EPS).sqrt()
        if s["gate"] is not None:
            z = s["gate"][rows].double().requires_grad_(grad)
            leaves.append(z)
            u = u * (torch.sigmoid(z) if case["gate"] == "sigmoid" else z)
        new = o["res_scale"] * x + o["branch_scale"] * u
        after = x if grad else new  # the gradient is given the residual after the block
        h = after / (after.pow(2).sum(-1, keepdim=True) / case["n"] + EPS).sqrt() * w_pre
        if not grad:
            blocks.append({"x": new, "h": h})
            continue
        dx, dw_pre = torch.autograd.grad(h, (x, w_pre), s["dh"][rows].double())
        dx = dx + s["dx"][rows].double()
        dy, dw_post, *dgate = torch.autograd.grad(new, leaves, dx)
        blocks.append({"dx": o["res_scale"] * dx, "dy": dy, **({"dgate": dgate[0]} if dgate else {})})
        weights[0] += dw_post
        weights[1] += dw_pre
    result = {name: torch.cat([x[name] for x in blocks]) for name in blocks[0]}
    return dict(result, dw_post=weights[0], dw_pre=weights[1]) if grad else result
