"""The biased attention at the framework's own lengths (documents of 256K tokens).

The bias gradient in closed form: with Q = 0 the probabilities depend on the
bias alone, P_ij = exp(b[u]) / Z_i for a distance in bucket u, and every sum over
a bucket's keys is a difference of prefix sums of V. dO_i and V_j turn with their
positions, so <dO_i, V_j> depends on the distance and a bucket's terms have one
sign: an error of a few percent in any bucket's sum shows.

And sampled rows of the 512K workload against the definition in 64 bits.
u = 2^-24 and h = 2^-11 are the half steps of fp32 and fp16."""
import math

import numpy as np
import pytest
import torch

import synth
from oracle import attention as A
from oracle import positions as N

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -11


def turning(T, wave):
    """[T, 2]: (cos, sin) of 2 pi t / wave, rounded to bf16."""
    t = torch.arange(T, dtype=torch.float64) * (2 * math.pi / wave)
    return torch.stack((torch.cos(t), torch.sin(t)), 1).to(torch.bfloat16)


def closed_form(b, starts, turn):
    """For each bucket: the gradient, the sum of P and the number of pairs; one head."""
    x = turn.double().numpy()
    T, i = len(x), np.arange(len(x))
    cum = np.concatenate([np.zeros((1, 2)), np.cumsum(x, 0)])
    ends = [min(int(e), T) for e in starts[1:]] + [T]
    hi = [np.maximum(i - int(s) + 1, 0) for s in starts]
    lo = [np.minimum(np.maximum(i - e + 1, 0), h) for e, h in zip(ends, hi)]
    w = np.exp(b - b.max())
    Z = sum(w[u] * (hi[u] - lo[u]) for u in range(len(w)))
    O = sum(w[u] * (cum[hi[u]] - cum[lo[u]]) for u in range(len(w))) / Z[:, None]
    D = (x * O).sum(1)
    out = []
    for u in range(len(w)):
        n = hi[u] - lo[u]
        s = (x * (cum[hi[u]] - cum[lo[u]])).sum(1) - D * n
        out.append(((w[u] * s / Z).sum(), (w[u] * n / Z).sum(), n.sum()))
    return np.array(out).T


def tolerance(mass, pairs, n):
    """|x| = |dP - D| <= 2.02 (bf16 rounds the turning vectors' norms up to 1 + 2^-8). dS = P x: P, x and the product in
    fp16 (3h), the scores' error twice (biases below 1, the exponential's 2^-21, LSE summed over n / 128 tiles in fp32).
    x: D is <dO, O>, |dO|_1 <= 1.42, and O has P in fp16 and n / 16 additions by the MMAs. The least of the scaled dS is
    2^-34 (dO's exponent 0, |V| < 2). The sum: a term goes through at most 2^14 additions."""
    es = 16 * U + 2.0 ** -21 + (n / 128 + 32) * U
    eO = H + 2 * es + n / 16 * 2 * U
    return mass * (2.02 * (3 * H + 2 * es + 2.0 ** 14 * U) + 1.42 * eO + 2.0 ** -22) + pairs * 2.0 ** -34


@pytest.mark.parametrize("T,wave", [(262144, 65536), (16385, 65536), (16385, 8192)])
def test_bias_gradient_in_closed_form(cuda, T, wave):
    from context_document_masked_gb300.session import CPAttention
    hq, hkv, d = 2, 1, 64
    # Inside the backward's table by distance, across its end (8192) and past it: wide buckets, and some of a distance or two.
    starts = [0, 1, 100, 700, 1500, 5000, 7700, 8180, 8200, 9000, 9003, 9004, 9040, 9041, 9300, 11000, 13000, 16300]
    starts += [20000, 30000, 45000, 56000, 75000, 120000, 130000, 200000, 262000] if T > 16385 else []
    b = 0.5 * torch.rand(hq, len(starts), generator=torch.Generator().manual_seed(3)) - 0.25
    turn = turning(T, wave)
    q, k = torch.zeros(T, hq, d, dtype=torch.bfloat16, device="cuda"), synth.make_qkv(T, hq, hkv, d, seed=1, device="cuda")[1]
    v, do = torch.zeros(T, hkv, d, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(q)
    v[:, 0, 5:7] = turn.cuda()
    do[:, :, 5:7] = turn.cuda()[:, None]
    s = CPAttention([T], 4, "perdoc", hq, hkv, d)
    s.gather(k, v)
    bc = b.cuda()
    out, lse = s.forward_bias(q, k, v, bc, starts, out_dtype=torch.float32)
    dq, dk, dv, db = s.backward_bias(q, k, v, out, lse, do, bc, starts)
    assert s.device_status() == 0 and (dk == 0).all()
    sharp = []
    for h in range(hq):
        want, mass, pairs = closed_form(b[h].double().numpy(), starts, turn)
        tol = tolerance(mass, pairs, T)
        assert (np.abs(db[h].double().cpu().numpy() - want) <= tol).all()
        sharp.append(tol <= 0.1 * np.abs(want))
    sharp = np.array(sharp)
    past = np.array(starts) >= 8192
    assert sharp.mean() >= 0.5 and sharp[:, past].mean() >= 0.4  # the check is able to fail, past the table too


def rows_of(q, k, v, do, b, starts, lo, rows, scale):
    """For query rows (local numbers) of a document at lo, all heads, in 64 bits on the GPU: O, LSE, dQ and their
    bounds [rows, hq, d] (LSE [rows, hq]), and P, dS with theirs for the keys.

    Bounds: independent roundings of terms, each at most e_j, make a sum off by 8 sqrt(sum e_j^2 / 3) at most (eight
    standard deviations); what all terms of a row share (LSE, D) counts whole; n additions of partial sums whose sizes
    add up to s are off by 2 u s."""
    n_max, (_, hq, d), hkv = max(rows) + 1, q.shape, k.shape[1]
    G = hq // hkv
    K, V = (x[lo:lo + n_max].double() for x in (k, v))
    start = torch.tensor(starts[1:], device="cuda")
    for r in rows:
        Q, dO, n = q[lo + r].double().view(hkv, G, d), do[lo + r].double().view(hkv, G, d), r + 1
        Kr, Vr = K[:n].transpose(0, 1), V[:n].transpose(0, 1)          # [hkv, n, d]
        bucket = torch.bucketize(torch.arange(r, -1, -1, device="cuda"), start, right=True)
        s = scale * Q @ Kr.transpose(1, 2) + b[:, bucket].double().view(hkv, G, n)
        lse = torch.logsumexp(s, -1, keepdim=True)
        p = torch.exp(s - lse)
        es = (d + 8) * 2 * U * scale * float((Q.abs() @ Kr.abs().transpose(1, 2)).max()) + 8 * U * float(b.abs().max()) + 2.0 ** -21
        es += (n / 128 + 32) * U                                         # LSE: additions over key tiles
        tiles = torch.nn.functional.pad(torch.einsum("kgn,knd->kgnd", p, Vr), (0, 0, 0, -n % 128)).view(hkv, G, -1, 128, d)
        parts = tiles.sum(3).cumsum(2).abs().sum(2) * 8                  # partial sums: eight MMAs a tile
        O = tiles.sum((2, 3))
        least = 2.0 ** -25 * torch.exp(s.amax(-1, keepdim=True) - lse)   # P beside V is relative to the row's largest
        eO = 8 / 3 ** 0.5 * (((H * p + least) ** 2) @ Vr ** 2).sqrt() + 2 * es * (p @ Vr.abs()) / n ** 0.5 * 8 + es * O.abs()
        eO = eO + 2 * U * parts
        del tiles
        x = dO @ Vr.transpose(1, 2) - (dO * O).sum(-1, keepdim=True)
        ds = p * x
        eD = (dO.abs() * eO).sum(-1, keepdim=True)                       # shared by the row's terms
        floor = 2.0 ** -24 * (1 + x.abs()) / 8                           # the least of the scaled dS and P (dO, V of a few units)
        # P, x and their product in fp16, the scores; dP's eight MMAs add to partial sums below 32 (2^-15 of P).
        e = (3 * H + 2 * es) * ds.abs() + 2.0 ** -15 * p + floor * 2.0 ** -8
        dQ = scale * ds @ Kr
        eQ = scale * (8 / 3 ** 0.5 * (e ** 2 @ Kr ** 2).sqrt() + eD * (p @ Kr).abs()) + es * dQ.abs()
        per = torch.nn.functional.pad(torch.einsum("kgn,knd->kgnd", ds, Kr), (0, 0, 0, -n % 128)).view(hkv, G, -1, 128, d).sum(3)
        eQ = eQ + scale * U * per.abs().sum(2) * (n // 128 + 1) ** 0.5 * 8  # reduce-adds of the key tiles, in any order
        yield r, (O, eO), (lse[..., 0], torch.full_like(lse[..., 0], es + 2.0 ** -20)), (dQ, eQ), (p, ds, e + p * eD)


def test_sampled_rows_of_the_512k_workload(cuda):
    from context_document_masked_gb300 import fcp
    from context_document_masked_gb300.session import CPAttention
    w, docs = synth.WORKLOADS[5], synth.doc_lengths(5)
    T, hq, hkv, d = w.T, w.Hq, w.Hkv, w.d
    G, scale = hq // hkv, 1 / math.sqrt(d)
    starts = fcp.rel_buckets(64, 100000).tolist()
    q, k, v = synth.make_qkv(T, hq, hkv, d, seed=2005, device="cuda")
    do = synth.make_dout(T, hq, d, seed=2005, device="cuda")
    b = torch.randn(hq, len(starts), generator=torch.Generator().manual_seed(5)).cuda()
    s = CPAttention(docs, w.cp, w.policy, hq, hkv, d)
    s.gather(k, v)
    out, lse = s.forward_bias(q, k, v, b, starts, out_dtype=torch.float32)
    dq, dk, dv, db = s.backward_bias(q, k, v, out, lse, do, b, starts)
    assert s.device_status() == 0
    cu, rng = synth.cu_from_lengths(docs), np.random.default_rng(5)
    order = np.argsort(docs)
    worst = {}

    def check(name, got, want, err):
        over = ((got.double() - want).abs() / err.clamp(min=1e-30)).max()
        worst[name] = max(worst.get(name, 0.0), float(over))

    for i in [order[-1], order[-2], order[len(order) // 2], order[0]]:
        lo, n = int(cu[i]), int(docs[i])
        rows = sorted({0, n - 3, n - 2, n - 1, *rng.integers(0, n, 2).tolist()} & set(range(n)))
        kp = {}
        for r, O, L, dQ, last in rows_of(q, k, v, do, b, starts, lo, rows, scale):
            check("O", out[lo + r].view(hkv, G, d), *O)
            check("LSE", lse[:, lo + r].view(hkv, G), *L)
            check("dQ", dq[lo + r].view(hkv, G, d), *dQ)
            if r >= n - 3:
                kp[r] = [t[..., max(0, n - 3):].cpu() for t in last]
            del last
        for j in range(max(0, n - 3), n):  # the last keys: seen by these rows alone
            dK = dV = eK = eV = 0
            for r in range(j, n):
                p, ds, e = (t[..., j - max(0, n - 3), None].cuda() for t in kp[r])
                Q, dO = q[lo + r].double().view(hkv, G, d), do[lo + r].double().view(hkv, G, d)
                dK, eK = dK + scale * (ds * Q).sum(1), eK + scale * (e * Q.abs()).sum(1)
                dV = dV + (p * dO).sum(1)
                # P in fp16 (its least 2^-35) and the scores, below another h; dO's least 2^-25 of a row's norm, below 16.
                eV = eV + ((2 * H * p + 2.0 ** -35) * dO.abs() + p * 2.0 ** -21).sum(1)
            check("dK", dk[lo + j], dK, eK)
            check("dV", dv[lo + j], dV, eV)
    print({n: round(x, 3) for n, x in worst.items()})
    assert set(worst) == {"O", "LSE", "dQ", "dK", "dV"} and max(worst.values()) <= 1, worst
    # The softmax's gradient over a row adds up to nothing, and so does each head's bias gradient.
    assert (db.double().sum(1).abs() <= 0.01 * db.double().abs().sum(1)).all()
