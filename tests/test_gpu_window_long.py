"""Windowed attention at the sizes of the workloads: sampled rows of the forward and of dQ
against the definition in 64 bits (bounds as in test_gpu_window.py), dK and dV of a
sample of keys from the rows that see them, and two sessions at once on two streams."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -11


def run(docs, cp, hq, hkv, d, window, sinks, seed, stream=None):
    from context_document_masked_gb300.session import CPAttention
    T = sum(docs)
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, do = (torch.randn(T, h, d, generator=g, device="cuda").bfloat16() for h in (hq, hkv, hkv, hq))
    s = CPAttention(docs, cp, "perdoc", hq, hkv, d, window=window, sinks=sinks)
    torch.cuda.synchronize()
    s.gather(k, v, stream=stream)
    out, lse = s.forward(q, k, v, out_dtype=torch.float32, stream=stream)
    return s, (q, k, v, do), (out, lse, *s.backward(q, k, v, out, lse, do, stream=stream))


def check(docs, window, sinks, x, got, rows, keys):
    q, k, v, do = x
    out, lse, dq, dk, dv = got
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    G, scale = hq // hkv, 1 / math.sqrt(d)
    T = q.shape[0]
    start = torch.repeat_interleave(torch.tensor([sum(docs[:i]) for i in range(len(docs))]), torch.tensor(docs)).tolist()
    es = (d + 8) * 2 * U * scale * 36 * d + 2.0 ** -21  # |q|, |k| < 6
    n = window + sinks

    def row(i, h):
        """Keys, probabilities and dS of a row, with its O, D and LSE."""
        a = start[i]
        key = torch.arange(a, i + 1, device="cuda")
        key = key[(i - key < window) | (key - a < sinks)]
        K, V = k[key, h // G].double(), v[key, h // G].double()
        s = scale * K @ q[i, h].double()
        p = torch.softmax(s, 0)
        o = p @ V
        dp = V @ do[i, h].double()
        return key, K, V, p, o, torch.logsumexp(s, 0), p * (dp - (p * dp).sum()), dp

    for i, h in rows:
        key, K, V, p, o, l, ds, dp = row(i, h)
        e_o = (H + 2 * es + n * 2 * U) * (p @ V.abs()) + n * 2.0 ** -25 * 6
        assert ((out[i, h].double() - o).abs() <= e_o).all()
        assert abs(lse[h, i].item() - l.item()) <= es + (n + 8) * 2 * U
        e_x = (d + 2) * 2 * U * (V.abs() @ do[i, h].double().abs()) + (do[i, h].double().abs() * e_o).sum()
        e_ds = (3 * H + 2 * es + n * 2 * U) * ds.abs() + p * e_x + 2.0 ** -24 * (1 + dp.abs() + (p * dp).sum().abs())
        assert ((dq[i, h].double() - scale * ds @ K).abs() <= scale * e_ds @ K.abs()).all()
    for j, g in keys:
        a = start[j]
        end = next((b for b in range(j, T + 1) if b == T or start[b] != a))
        ref_k, err_k, ref_v, err_v = (torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(4))
        last = end if j - a < sinks else min(end, j + window)
        count = (last - j) * G
        for h in range(g * G, (g + 1) * G):
            for i in range(j, last):
                key, K, V, p, o, l, ds, dp = row(i, h)
                c = (key == j).nonzero()[0, 0]
                Q, dO = q[i, h].double(), do[i, h].double()
                e_o = (H + 2 * es + n * 2 * U) * (p @ V.abs()) + n * 2.0 ** -25 * 6
                e_x = (d + 2) * 2 * U * (V[c].abs() @ dO.abs()) + (dO.abs() * e_o).sum()
                e_ds = (3 * H + 2 * es + count * 2 * U) * ds[c].abs() + p[c] * e_x + 2.0 ** -24 * (1 + (dp[c] - (p * dp).sum()).abs())
                ref_k += scale * ds[c] * Q
                err_k += scale * e_ds * Q.abs()
                ref_v += p[c] * dO
                err_v += (H + 2 * es + count * 2 * U) * p[c] * dO.abs() + 2.0 ** -24 * dO.abs()
        assert ((dk[j, g].double() - ref_k).abs() <= err_k).all()
        assert ((dv[j, g].double() - ref_v).abs() <= err_v).all()


@pytest.mark.parametrize("docs,cp,hq,hkv,d,window,sinks,far", [
    ([65536], 8, 16, 2, 128, 2048, 16, False),
    ([30000, 1, 2767], 4, 12, 12, 64, 256, 4, True),
    ([20000, 12768], 16, 32, 8, 128, 128, 0, False)])
def test_sampled_rows(cuda, docs, cp, hq, hkv, d, window, sinks, far):
    T = sum(docs)
    s, x, got = run(docs, cp, hq, hkv, d, window, sinks, seed=T)
    assert s.device_status() == 0
    r = torch.Generator().manual_seed(1)
    picks = torch.randint(T, (40,), generator=r).tolist() + [0, window - 1, window, window + sinks, T - 1]
    rows = [(i, int(torch.randint(hq, (1,), generator=r))) for i in picks]
    # Keys with few rows that see them, so that the sum over rows stays short; a sink only where asked for.
    keys = [(T - 1, 0), (T - 40, hkv - 1), (docs[0] - 3, 0)]
    if far:
        keys.append((T - docs[-1] + 1, 1))  # a sink of the last document
    check(docs, window, sinks, x, got, rows, keys)


def test_two_sessions_at_once(cuda):
    """Two streams, each with its session, workspace and window."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    made = [run([9000, 3000], 4, 8, 2, 128, w, sk, seed=w, stream=st) for st, (w, sk) in zip(streams, ((128, 4), (700, 0)))]
    torch.cuda.synchronize()
    for (s, x, got), (w, sk) in zip(made, ((128, 4), (700, 0))):
        assert s.device_status() == 0
        check([9000, 3000], w, sk, x, got, [(i, i % 8) for i in range(0, 12000, 397)], [(11990, 1)])
