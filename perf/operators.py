"""Workloads of the position operators around document-masked attention.

Two operators, each with its gradient, over a packed sequence whose documents
fix the positions (a document's first token has position 0):

  norm_rope       RMS norm of every query and key head and the rotary rotation
                  by the position inside the document, from the fused
                  projection of a layer to the contiguous Q, K and V that the
                  attention reads.
  norm_rope_grad  its gradient: from the attention's fp32 dQ, dK and dV to the
                  gradient of the fused projection and of the norm weights.
  bias_attn       document-masked attention with a learned bias for each head
                  and bucket of the distance i - j.
  bias_attn_step  the same forward and its gradients, that of the bias table
                  among them.

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
        # Norm and rotation. The small sequence of 4 query and 2 KV heads: a call that is all latency.
        dict(name="norm_rope 2k h4 d64", op="norm_rope", T=2048, hq=4, hkv=2, d=64, rot=64, interleaved=False,
             theta=1e4, docs="uniform 64 640", doc_seed=1, cp=2, policy="llama3"),
        # A ragged batch: odd length, few heads, half of each head rotated, neighbouring pairs.
        dict(name="norm_rope 5003 h6 rot64", op="norm_rope", T=5003, hq=6, hkv=2, d=128, rot=64, interleaved=True,
             theta=1e4, docs="lognormal 5.0 1.2 1 2048", doc_seed=2, cp=1, policy="perdoc"),
        # Short documents with a few long ones at 64 query heads, all 16 shards at once: the largest.
        dict(name="norm_rope 64k h64", op="norm_rope", T=65536, hq=64, hkv=8, d=128, rot=128, interleaved=False,
             theta=5e5, docs="mix 128 1024 4096 16384", doc_seed=4, cp=16, policy="wholedoc"),
        dict(name="norm_rope_grad 2k h4 d64", op="norm_rope_grad", T=2048, hq=4, hkv=2, d=64, rot=64,
             interleaved=False, theta=1e4, docs="uniform 64 640", doc_seed=1, cp=2, policy="llama3"),
        dict(name="norm_rope_grad 5003 h6 rot64", op="norm_rope_grad", T=5003, hq=6, hkv=2, d=128, rot=64,
             interleaved=True, theta=1e4, docs="lognormal 5.0 1.2 1 2048", doc_seed=2, cp=1, policy="perdoc"),
        # The 32K packed sequence of a 32/8-head layer, one training step's share.
        dict(name="norm_rope_grad 32k h32", op="norm_rope_grad", T=32768, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, theta=5e5, docs="lognormal 7.5 1.2 32 32768", doc_seed=1002, cp=4, policy="perdoc"),
        # Attention with a bias of 32 buckets up to distance 128 (exact to 16, then spaced by logarithms).
        dict(name="bias_attn 2k h4 d64", op="bias_attn", T=2048, hq=4, hkv=2, d=64, buckets=32, reach=128,
             docs="uniform 64 640", doc_seed=1, cp=2, policy="llama3"),
        dict(name="bias_attn 32k h32", op="bias_attn", T=32768, hq=32, hkv=8, d=128, buckets=32, reach=128,
             docs="lognormal 7.5 1.2 32 32768", doc_seed=1002, cp=4, policy="perdoc"),
        # Training steps: short documents and as many KV as query heads ...
        dict(name="bias_attn_step 4k h12 d64", op="bias_attn_step", T=4096, hq=12, hkv=12, d=64, buckets=32, reach=128,
             docs="uniform 64 640", doc_seed=3, cp=2, policy="perdoc"),
        # ... an odd length, groups of three heads, buckets that reach far ...
        dict(name="bias_attn_step 7001 h6", op="bias_attn_step", T=7001, hq=6, hkv=2, d=128, buckets=48, reach=2000,
             docs="lognormal 6.5 1.2 1 4096", doc_seed=5, cp=1, policy="perdoc"),
        # ... one long document cut over eight shards ...
        dict(name="bias_attn_step 16k h16", op="bias_attn_step", T=16384, hq=16, hkv=2, d=128, buckets=64, reach=8192,
             docs="one", doc_seed=6, cp=8, policy="perdoc"),
        # ... and the 32K packed sequence: the largest.
        dict(name="bias_attn_step 32k h32", op="bias_attn_step", T=32768, hq=32, hkv=8, d=128, buckets=32, reach=128,
             docs="lognormal 7.5 1.2 32 32768", doc_seed=1002, cp=4, policy="perdoc"),
    ]


HEADS = [(4, 2, 64), (5, 5, 64), (8, 1, 64), (12, 12, 64), (6, 2, 128), (16, 2, 128), (32, 8, 128), (64, 8, 128)]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "bias_attn", "bias_attn_step"])
    hq, hkv, d = rng.choice(HEADS)
    rope = op.startswith("norm_rope")
    low = 64 if op == "bias_attn_step" else 1  # a document of one token has no gradient of Q, K and the bias
    c = dict(op=op, T=_log_uniform(rng, low, 65536 if rope else 32768), hq=hq, hkv=hkv, d=d,
             docs=rng.choice(["one", "uniform 64 640", "uniform 1 200", "lognormal 5.0 1.2 1 2048",
                              "lognormal 7.5 1.2 32 32768", "mix 128 1024 4096 16384"]),
             doc_seed=rng.randrange(1 << 20), cp=rng.choice([1, 2, 4, 8]), policy="perdoc")
    if rope:
        c.update(rot=rng.choice([0, 16, 32, d // 2, d, d]), interleaved=rng.random() < 0.5,
                 theta=rng.choice([1e4, 5e5]))
    else:
        c.update(buckets=rng.choice([8, 17, 32, 48, 64]), reach=_log_uniform(rng, 64, 8192))
    most = max((x for x in listed() if x["op"] == op), key=lambda x: max(work(x)["flops"], work(x)["bytes"]))
    most, longest = work(most), 16 * 16384 ** 2  # the plain form holds one document's scores of every head
    while work(c)["flops"] > most["flops"] or work(c)["bytes"] > most["bytes"] or (
            not rope and hq * max(doc_lengths(c)) ** 2 > longest):
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


def bucket_starts(buckets, reach):
    """First distance of each bucket: one bucket a distance up to half of them, then spaced by logarithms up to `reach`."""
    exact = buckets // 2
    far = [math.ceil(exact * (reach / exact) ** (k / (buckets - exact))) for k in range(buckets - exact)]
    return [int(x) for x in np.maximum.accumulate(list(range(exact)) + far)]


def work(case):
    T, hq, hkv, d = case["T"], case["hq"], case["hkv"], case["d"]
    heads, n = hq + 2 * hkv, case["T"] * (hq + hkv) * case["d"]
    if case["op"] == "norm_rope":
        return {"bytes": 2 * T * heads * d * 2 + 8 * d, "flops": 10 * n}
    if case["op"] == "norm_rope_grad":  # fp32 gradients and the projection's Q and K in, bf16 gradients out
        return {"bytes": T * heads * d * (4 + 2) + T * (hq + hkv) * d * 2 + 16 * d, "flops": 24 * n}
    pairs = sum(L * (L + 1) // 2 for L in doc_lengths(case))
    table = hq * case["buckets"] * 4
    if case["op"] == "bias_attn":
        return {"bytes": T * (2 * hq + 2 * hkv) * d * 2 + hq * T * 4 + table, "flops": 4 * d * hq * pairs}
    return {"bytes": T * (4 * hq + 4 * hkv) * d * 2 + hq * T * 4 + 2 * table, "flops": 14 * d * hq * pairs}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    T, hq, hkv, d = case["T"], case["hq"], case["hkv"], case["d"]
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    lengths = doc_lengths(case)
    s = dict(case=case, lengths=lengths, session=None)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    if case["op"].startswith("norm_rope"):
        s["qkv"] = normal(T, hq + 2 * hkv, d)  # the fused projection
        s["wq"] = 1 + 0.1 * normal(d, dtype=torch.float32)
        s["wk"] = 1 + 0.1 * normal(d, dtype=torch.float32)
        rot = case["rot"]
        s["inv_freq"] = case["theta"] ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / max(rot, 1))
        s["inv_freq"] = s["inv_freq"].float() if rot else None
        first = np.concatenate([[0], np.cumsum(lengths)[:-1]])
        s["position"] = torch.from_numpy(np.arange(T) - np.repeat(first, lengths)).to(dev)
        if case["op"] == "norm_rope_grad":
            s["dq"] = normal(T, hq, d, dtype=torch.float32)
            s["dk"] = normal(T, hkv, d, dtype=torch.float32)
            s["dv"] = normal(T, hkv, d, dtype=torch.float32)
    else:
        s["q"], s["k"], s["v"] = normal(T, hq, d), normal(T, hkv, d), normal(T, hkv, d)
        s["bias"] = normal(hq, case["buckets"], dtype=torch.float32)
        s["starts"] = bucket_starts(case["buckets"], case["reach"])
        if case["op"] == "bias_attn_step":
            s["do"] = normal(T, hq, d)
    if own:
        from context_document_masked_gb300.session import CPAttention

        s["session"] = CPAttention(lengths, case["cp"], case["policy"], hq, hkv, d, device=dev)
    return s


# --------------------------------------------------------------- operators


def run(s):
    op = s["case"]["op"]
    if op == "norm_rope":
        return own_norm_rope(s) if own else plain_norm_rope(s)
    if op == "norm_rope_grad":
        return own_norm_rope_grad(s) if own else plain_norm_rope_grad(s)
    return own_bias_attn(s) if own else plain_bias_attn(s)


def own_norm_rope(s):
    hq, hkv, qkv = s["case"]["hq"], s["case"]["hkv"], s["qkv"]
    q, k, v = s["session"].qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], wq=s["wq"], wk=s["wk"],
                                        inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"], eps=EPS)
    return {"q": q, "k": k, "v": v}


def own_norm_rope_grad(s):
    hq, hkv, qkv = s["case"]["hq"], s["case"]["hkv"], s["qkv"]
    dqkv = torch.empty_like(qkv)
    *_, dwq, dwk = s["session"].qk_norm_rope_backward(
        s["dq"], s["dk"], s["dv"], qkv[:, :hq], qkv[:, hq:hq + hkv], wq=s["wq"], wk=s["wk"], inv_freq=s["inv_freq"],
        interleaved=s["case"]["interleaved"], eps=EPS, dq_in=dqkv[:, :hq], dk_in=dqkv[:, hq:hq + hkv],
        dv_in=dqkv[:, hq + hkv:])
    return {"dqkv": dqkv, "dwq": dwq, "dwk": dwk}


def own_bias_attn(s):
    a, q, k, v, bias, starts = s["session"], s["q"], s["k"], s["v"], s["bias"], s["starts"]
    a.gather(k, v)
    if s["case"]["op"] == "bias_attn":
        out, lse = a.forward_bias(q, k, v, bias, starts)
        return {"out": out, "lse": lse}
    out, lse = a.forward_bias(q, k, v, bias, starts, out_dtype=torch.float32)
    grads = a.backward_bias(q, k, v, out, lse, s["do"], bias, starts)
    # The next layers take bf16, the type of the tensors that these are the gradients of.
    return dict(zip(("out", "dq", "dk", "dv", "dbias"), (x.to(torch.bfloat16) for x in (out, *grads))), lse=lse)


def angles(s):
    """cos and sin of position * inv_freq, [T, 1, rot / 2]: far positions times a frequency need 64 bits."""
    a = s["position"].double()[:, None, None] * s["inv_freq"].double()
    return a.cos().float(), a.sin().float()


def turn(x, cos, sin, interleaved):
    """The leading 2 * cos.shape[-1] dimensions of x rotated by the pair angles."""
    n = cos.shape[-1]
    pairs = x[..., :2 * n]
    a, b = (pairs[..., 0::2], pairs[..., 1::2]) if interleaved else (pairs[..., :n], pairs[..., n:])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., 2 * n:]), -1)


def plain_norm_rope(s):
    hq, hkv, inter = s["case"]["hq"], s["case"]["hkv"], s["case"]["interleaved"]

    def one(x, w):
        x = x.float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        if s["inv_freq"] is not None:
            y = turn(y, *angles(s), inter)
        return y.to(torch.bfloat16)

    qkv = s["qkv"]
    return {"q": one(qkv[:, :hq], s["wq"]), "k": one(qkv[:, hq:hq + hkv], s["wk"]), "v": qkv[:, hq + hkv:].clone()}


def plain_norm_rope_grad(s):
    hq, hkv, inter = s["case"]["hq"], s["case"]["hkv"], s["case"]["interleaved"]

    def one(x, w, dy):
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        if s["inv_freq"] is not None:
            cos, sin = angles(s)
            dy = turn(dy, cos, -sin, inter)
        xn = x * r
        g = dy * w
        return r * (g - xn * (g * xn).mean(-1, keepdim=True)), (dy * xn).sum((0, 1))

    qkv = s["qkv"]
    dxq, dwq = one(qkv[:, :hq], s["wq"], s["dq"])
    dxk, dwk = one(qkv[:, hq:hq + hkv], s["wk"], s["dk"])
    return {"dqkv": torch.cat((dxq, dxk, s["dv"]), 1).to(torch.bfloat16), "dwq": dwq, "dwk": dwk}


def plain_bias_attn(s):
    case = s["case"]
    hq, hkv, d, G = case["hq"], case["hkv"], case["d"], case["hq"] // case["hkv"]
    scale, grad = 1 / math.sqrt(case["d"]), case["op"] == "bias_attn_step"
    starts = torch.tensor(s["starts"], device="cuda")
    dbias = torch.zeros_like(s["bias"])
    outs, at = [], 0
    for n in s["lengths"]:  # nothing passes between documents: each is a causal attention of its own
        q, k, v = (s[x][at:at + n].float().transpose(0, 1) for x in "qkv")
        k, v = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
        distance = torch.arange(n, device="cuda")[:, None] - torch.arange(n, device="cuda")
        bucket = torch.searchsorted(starts, distance.clamp(min=0), right=True) - 1
        p = (q @ k.transpose(1, 2)).mul_(scale).add_(s["bias"][:, bucket]).masked_fill_(distance < 0, -math.inf)
        m = p.amax(-1, keepdim=True)
        p = p.sub_(m).exp_()
        l = p.sum(-1, keepdim=True)
        p = p.div_(l)
        out = p @ v
        one = [out, (m + l.log())[..., 0]]
        if grad:
            do = s["do"][at:at + n].float().transpose(0, 1)
            ds = (do @ v.transpose(1, 2)).sub_((do * out).sum(-1, keepdim=True)).mul_(p)
            dq = (ds @ k).mul_(scale)
            dk = (ds.transpose(1, 2) @ q).mul_(scale).view(hkv, G, n, d).sum(1)
            dv = (p.transpose(1, 2) @ do).view(hkv, G, n, d).sum(1)
            # Sums along the diagonals: in rows of n + 1 elements, distance x falls into column -x.
            by = torch.nn.functional.pad(ds.reshape(hq, n * n), (0, n)).view(hq, n, n + 1).sum(1)
            by = torch.cat((by[:, :1], by[:, 2:].flip(1)), 1)
            dbias.index_add_(1, bucket[:, 0], by)
            one += [dq, dk, dv]
        outs.append(one)
        at += n
    out, lse, *g = (torch.cat([o[i] for o in outs], 1) for i in range(len(outs[0])))
    lse = lse.contiguous()
    if not grad:
        return {"out": out.transpose(0, 1).to(torch.bfloat16), "lse": lse}
    dq, dk, dv = (x.transpose(0, 1).to(torch.bfloat16) for x in g)
    return {"out": out.transpose(0, 1).to(torch.bfloat16), "lse": lse, "dq": dq, "dk": dk, "dv": dv,
            "dbias": dbias.to(torch.bfloat16)}


# ------------------------------------------------------- 64-bit definitions


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm_rope"):
        return exact_norm_rope(s)
    if work(case)["flops"] > 1.2e13:  # over what the 64-bit units do in the time there is
        return None
    return exact_bias_attn(s)


def exact_norm_rope(s):
    """By complex multiplication; the gradient by automatic differentiation."""
    case = s["case"]
    hq, hkv, d, rot = case["hq"], case["hkv"], case["d"], case["rot"]
    grad = case["op"] == "norm_rope_grad"

    def one(x, w, dy):
        x, w = x.double().requires_grad_(grad), w.double().requires_grad_(grad)
        y = x / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w
        if rot:
            a = torch.outer(s["position"].double(), s["inv_freq"].double())
            unit = torch.complex(torch.cos(a), torch.sin(a))[:, None]
            z = y[..., :rot].unflatten(-1, (rot // 2, 2) if case["interleaved"] else (2, rot // 2))
            z = z if case["interleaved"] else z.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * unit)
            z = z if case["interleaved"] else z.transpose(-1, -2)
            y = torch.cat((z.flatten(-2), y[..., rot:]), -1)
        return torch.autograd.grad(y, (x, w), dy.double()) if grad else y

    qkv = s["qkv"]
    dy = (s["dq"], s["dk"]) if grad else (None, None)
    q, k = one(qkv[:, :hq], s["wq"], dy[0]), one(qkv[:, hq:hq + hkv], s["wk"], dy[1])
    if not grad:
        return {"q": q, "k": k, "v": qkv[:, hq + hkv:].double()}
    return {"dqkv": torch.cat((q[0], k[0], s["dv"].double()), 1), "dwq": q[1], "dwk": k[1]}


def exact_bias_attn(s):
    """One head and one block of query rows at a time, against the keys up to the block's end."""
    case = s["case"]
    T, hq, hkv, d = case["T"], case["hq"], case["hkv"], case["d"]
    G, grad = hq // hkv, case["op"] == "bias_attn_step"
    new = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros(T, hq, d, **new), torch.zeros(hq, T, **new)
    dq, dk, dv = torch.zeros(T, hq, d, **new), torch.zeros(T, hkv, d, **new), torch.zeros(T, hkv, d, **new)
    dbias = torch.zeros(hq, case["buckets"], **new)
    edges = torch.tensor(s["starts"][1:], device="cuda")
    step = 1024
    at = 0
    for n in s["lengths"]:
        for a in range(at, at + n, step):
            b = min(a + step, at + n)
            dist = torch.arange(a, b, device="cuda")[:, None] - torch.arange(at, b, device="cuda")
            seen = dist >= 0
            bucket = torch.bucketize(dist.clamp(min=0), edges, right=True)
            for h in range(hq):
                q, k, v = s["q"][a:b, h].double(), s["k"][at:b, h // G].double(), s["v"][at:b, h // G].double()
                x = torch.where(seen, q @ k.T / math.sqrt(d) + s["bias"][h].double()[bucket], -math.inf)
                y = torch.logsumexp(x, 1)
                p = torch.exp(x - y[:, None])
                o = p @ v
                out[a:b, h], lse[h, a:b] = o, y
                if grad:
                    do = s["do"][a:b, h].double()
                    dp = do @ v.T
                    ds = p * (dp - (p * dp).sum(1, keepdim=True))
                    dq[a:b, h] = ds @ k / math.sqrt(d)
                    dk[at:b, h // G] += ds.T @ q / math.sqrt(d)
                    dv[at:b, h // G] += p.T @ do
                    # One sum for each distance, then one for each bucket.
                    m = b - at
                    lines = torch.zeros(b - a, m + 1, **new)
                    lines[:, :m] = ds.flip(1)
                    lines = torch.nn.functional.pad(lines, (0, b - a)).flatten()[:(b - a) * (m + b - a)]
                    lines = lines.view(b - a, m + b - a).sum(0)  # column c: key index m - 1 - c + row, distance c - rows + 1
                    dbias[h].index_add_(0, bucket[-1].flip(0), lines[b - a - 1:b - a - 1 + m])
        at += n
    if not grad:
        return {"out": out, "lse": lse}
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv, "dbias": dbias}
