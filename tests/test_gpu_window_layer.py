"""A sliding-window layer as a program runs it, forward and backward: the norm
before the block, the projection, head norm and rotation, windowed attention, the
output projection, the norm behind the block with its gate and the sum with the
residual; against the same layer in 64 bits with automatic differentiation."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_layer(cuda):
    from context_document_masked_gb300.session import CPAttention
    docs, hq, hkv, d, window, sinks = [300, 1, 211, 88], 4, 2, 64, 96, 4
    T, n = sum(docs), hq * d
    heads = hq + 2 * hkv
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)
    x, dout, dres = normal(T, n), normal(T, n, scale=0.5), normal(T, n, scale=0.5)
    w_in, w_out = normal(n, heads * d + n, scale=n ** -0.5), normal(n, n, scale=n ** -0.5)
    ws = [1 + 0.1 * normal(k, dtype=torch.float32) for k in (n, d, d, n, n)]  # before, q, k, behind, next
    inv_freq = 1e4 ** (-torch.arange(0, d, 2, device="cuda") / d)
    s = CPAttention(docs, 2, "perdoc", hq, hkv, d, window=window, sinks=sinks)
    scales = dict(res_scale=0.9, branch_scale=0.7)

    # Forward.
    _, h = s.residual_norm(x, w_pre=ws[0])
    fused = h @ w_in
    qkv, gate = fused[:, :heads * d].view(T, heads, d), fused[:, heads * d:]
    slices = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    q, k, v = s.qk_norm_rope(*slices, wq=ws[1], wk=ws[2], inv_freq=inv_freq)
    s.gather(k, v)
    o, lse = s.forward(q, k, v, out_dtype=torch.float32)
    o16 = o.bfloat16()
    y = o16.view(T, n) @ w_out
    x2, h2 = s.residual_norm(x, y, gate, w_post=ws[3], w_pre=ws[4], **scales)

    # Backward, into one fused gradient of the projection.
    dx, dy, dgate, dw3, dw4 = s.residual_norm_backward(dout, dres, x2, y, gate, w_post=ws[3], w_pre=ws[4], **scales)
    dw_out = o16.view(T, n).t() @ dy
    dq, dk, dv = s.backward(q, k, v, o, lse, (dy @ w_out.t()).view(T, hq, d))
    dfused = torch.empty_like(fused)
    dqkv = dfused[:, :heads * d].view(T, heads, d)
    dfused[:, heads * d:] = dgate
    *_, dw1, dw2 = s.qk_norm_rope_backward(dq, dk, dv, slices[0], slices[1], wq=ws[1], wk=ws[2], inv_freq=inv_freq,
                                           dq_in=dqkv[:, :hq], dk_in=dqkv[:, hq:hq + hkv], dv_in=dqkv[:, hq + hkv:])
    dw_in = h.t() @ dfused
    dx, *_, dw0 = s.residual_norm_backward(dfused @ w_in.t(), dx, x, w_pre=ws[0])
    assert s.device_status() == 0

    # The same in 64 bits.
    D = [t.double().requires_grad_() for t in (x, w_in, w_out, *ws)]
    x64, i64, o64, *w64 = D

    def norm(t, w):
        return t * torch.rsqrt(t.pow(2).mean(-1, keepdim=True) + 1e-6) * w
    f = norm(x64, w64[0]) @ i64
    parts, gz = f[:, :heads * d].view(T, heads, d), f[:, heads * d:]
    pos = torch.cat([torch.arange(m) for m in docs]).cuda().double()
    start = torch.arange(T, device="cuda") - pos.long()
    ang = pos[:, None, None] * inv_freq.double()

    def turned(t):
        a, b = t[..., :d // 2], t[..., d // 2:]
        return torch.cat((a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()), -1)
    Q, K = turned(norm(parts[:, :hq], w64[1])), turned(norm(parts[:, hq:hq + hkv], w64[2]))
    K, V = (t.repeat_interleave(hq // hkv, 1) for t in (K, parts[:, hq + hkv:]))
    i, j = torch.arange(T, device="cuda")[:, None], torch.arange(T, device="cuda")
    seen = (start[:, None] == start) & (j <= i) & ((i - j < window) | (j - start[:, None] < sinks))
    sc = torch.einsum("ihd,jhd->hij", Q, K) / math.sqrt(d)
    O = torch.einsum("hij,jhd->ihd", torch.softmax(sc.masked_fill(~seen, -torch.inf), -1), V)
    X2 = 0.9 * x64 + 0.7 * torch.sigmoid(gz) * norm(O.reshape(T, n) @ o64, w64[3])
    H2 = norm(X2, w64[4])
    grads = torch.autograd.grad((H2 * dout.double()).sum() + (X2 * dres.double()).sum(), D)

    # Every activation between the operators is bf16, off by 2^-9 to 2^-8 of its size. A dozen of them lie one behind
    # another on the longest path; their errors are independent, so in the norm of a whole tensor they add like
    # sqrt(12) 2^-8 / sqrt(3) of the values that meet there, and a norm's Jacobian or a softmax row can bring out
    # of them a few times the share of what remains.
    def off(a, b):
        return ((a.double() - b).norm() / b.norm()).item()
    assert off(x2, X2) < 2.0 ** -7 and off(h2, H2) < 2.0 ** -7
    for a, b in zip((dx, dw_in, dw_out, dw0, dw1, dw2, dw3, dw4), grads):
        assert off(a, b) < 2.0 ** -5
