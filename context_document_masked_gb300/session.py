"""One packed sequence, one CP plan, all shards on one GPU.

Holds the device copies of a plan's work tables and the buffers the C-ABI
calls need (received-key buffers, workspace), allocated once through PyTorch.
Every step of the path runs in libfcp; this class only orders the calls.
"""
from __future__ import annotations

import torch

from . import fcp


def _on_stream(stream):
    """The stream of a call (a torch stream, a raw handle or None: the current
    one) as a context: what torch does for the call runs in its order."""
    if stream is None:
        return fcp._HERE_CTX
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)


class CPAttention:
    def __init__(self, doclens, cp: int, policy: str, hq: int, hkv: int, d: int,
                 device="cuda", target_imbalance: float = 1.05, scale: float = 0.0, window: int = 0, sinks: int = 0):
        """window > 0: gather(), forward() and backward() are those of a sliding
        window (a token sees the last `window` tokens of its document, itself
        among them, and the document's first `sinks`). Sessions of one packed
        sequence that differ in their windows have the same shards."""
        self.device = torch.device(device)
        self.window, self.sinks = window, sinks
        self.plan = self._make_plan(doclens, cp, policy, target_imbalance)
        self.T = int(sum(int(x) for x in doclens))
        self.hq, self.hkv, self.d, self.cp = hq, hkv, d, cp
        self.scale = scale
        nbytes = self.plan.device_bytes()
        self.plan_buf = torch.empty(nbytes // 4, dtype=torch.int32, device=self.device)
        self.dplan = self.plan.upload(self.plan_buf)
        rows = max(1, self.dplan.total_remote_rows)
        self.kbuf = torch.empty(rows, hkv, d, dtype=torch.bfloat16, device=self.device)
        self.vbuf = torch.empty_like(self.kbuf)
        self.dims = fcp.dims(self.T, hq, hkv, d, scale)
        ws_bytes = fcp.workspace_bytes(self.dims, self.plan)
        self.ws = torch.zeros(ws_bytes // 4, dtype=torch.int32, device=self.device)

    def _make_plan(self, doclens, cp, policy, target_imbalance):
        if not self.window and self.sinks:
            raise ValueError("sinks are those of a window: window > 0")
        plan = fcp.Plan(doclens, cp, policy, target_imbalance)
        return plan.windowed(self.window, self.sinks) if self.window else plan

    def set_plan(self, doclens, target_imbalance: float = 1.05, stream=None):
        """A new plan for the next packed sequence (same T, CP size, policy,
        shapes and window), uploaded into this session's plan buffer on `stream`; the
        received-key buffers and the workspace are kept when they are large
        enough and replaced otherwise, in that stream's order. The previous plan's tables must no longer
        be in use by queued work on other streams."""
        if int(sum(int(x) for x in doclens)) != self.T:
            raise ValueError("set_plan: the token count differs from the session's")
        plan = self._make_plan(doclens, self.cp, self.plan.policy, target_imbalance)
        nbytes = plan.device_bytes()
        with _on_stream(stream):
            if self.plan_buf.numel() * 4 < nbytes:
                self.plan_buf = torch.empty(nbytes // 4, dtype=torch.int32, device=self.device)
            self.plan = plan
            self.dplan = plan.upload(self.plan_buf, stream=stream)
            rows = max(1, self.dplan.total_remote_rows)
            if self.kbuf.shape[0] < rows:
                self.kbuf = torch.empty(rows, self.hkv, self.d, dtype=torch.bfloat16, device=self.device)
                self.vbuf = torch.empty_like(self.kbuf)
            ws_bytes = fcp.workspace_bytes(self.dims, plan)
            if self.ws.numel() * 4 < ws_bytes:
                self.ws = torch.zeros(ws_bytes // 4, dtype=torch.int32, device=self.device)
        return self.dplan

    def stats(self) -> dict:
        return self.plan.stats()

    def gather(self, k, v, shard: int = -1, stream=None):
        fcp.gather_kv(k, v, self.dplan, shard, self.kbuf, self.vbuf, stream)

    def _out_lse(self, out, lse, out_dtype, stream):
        """The given tensors, or new ones made in the order of the call's stream."""
        with _on_stream(stream):
            if out is None:
                out = torch.empty(self.T, self.hq, self.d, dtype=out_dtype, device=self.device)
            if lse is None:
                lse = torch.empty(self.hq, self.T, dtype=torch.float32, device=self.device)
        return out, lse

    def forward(self, q, k, v, shard: int = -1, out=None, lse=None, kv_block=None,
                out_dtype=torch.bfloat16, stream=None):
        out, lse = self._out_lse(out, lse, out_dtype, stream)
        lo, hi = (0, self.T) if kv_block is None else kv_block
        fcp.attn_fwd(q, k, v, self.kbuf, self.vbuf, self.dplan, shard, out, lse, self.ws,
                     kv_lo=lo, kv_hi=hi, scale=self.scale, stream=stream)
        return out, lse

    def forward_qk8(self, q, k, v, shard: int = -1, out=None, lse=None, kv_block=None,
                    out_dtype=torch.bfloat16, stream=None):
        """forward() with Q K^T on e4m3 copies of Q and K (d = 128)."""
        out, lse = self._out_lse(out, lse, out_dtype, stream)
        lo, hi = (0, self.T) if kv_block is None else kv_block
        fcp.attn_fwd_qk8(q, k, v, self.kbuf, self.vbuf, self.dplan, shard, out, lse, self.ws,
                         kv_lo=lo, kv_hi=hi, scale=self.scale, stream=stream)
        return out, lse

    def forward_ring(self, q, k, v, ring_step: int = -1, shard: int = -1, out=None, lse=None,
                     out_dtype=torch.bfloat16, stream=None):
        """Forward in ring order without the gathered buffer: ring_step -1 visits
        every owner's keys in one pass, s >= 0 gives ring step s's partial."""
        out, lse = self._out_lse(out, lse, out_dtype, stream)
        fcp.attn_fwd_ring(q, k, v, self.dplan, shard, ring_step, out, lse, self.ws, scale=self.scale,
                          stream=stream)
        return out, lse

    def forward_bias(self, q, k, v, bias, starts, shard: int = -1, out=None, lse=None, kv_block=None,
                     out_dtype=torch.bfloat16, stream=None):
        """forward() with the learned bias[h, bucket(i - j)] (fp32 [hq][buckets])
        added to the scores; starts: the buckets' first distances (host), for
        instance fcp.rel_buckets(n, max_distance)."""
        out, lse = self._out_lse(out, lse, out_dtype, stream)
        lo, hi = (0, self.T) if kv_block is None else kv_block
        fcp.attn_fwd_bias(q, k, v, self.kbuf, self.vbuf, bias, starts, self.dplan, shard, out, lse, self.ws, kv_lo=lo,
                          kv_hi=hi, scale=self.scale, stream=stream)
        return out, lse

    def backward_bias(self, q, k, v, out, lse, dout, bias, starts, shard: int = -1, dq=None, dk=None, dv=None,
                      dbias=None, zero_grads: bool | None = None, stream=None):
        """backward() of forward_bias(); also returns the bias's gradient. zero_grads:
        dk, dv and dbias are set to zero first (all of their rows), else added to.
        It may be left out (then they are set to zero) but for one shard's call
        with given dk, dv or dbias: in a loop over shards that would keep the last
        one's share."""
        if zero_grads is None:
            if shard >= 0 and not (dk is None and dv is None and dbias is None):
                raise ValueError("backward_bias: one shard's gradients into given tensors: zero_grads says whether they "
                                 "are set to zero first (True) or added to (False)")
            zero_grads = True
        with _on_stream(stream):
            if dq is None:
                dq = torch.empty(self.T, self.hq, self.d, dtype=torch.float32, device=self.device)
            make = torch.empty if zero_grads else torch.zeros
            dk, dv = (make(self.T, self.hkv, self.d, dtype=torch.float32, device=self.device) if x is None else x
                      for x in (dk, dv))
            if dbias is None:
                dbias = make(bias.shape, dtype=torch.float32, device=self.device)
        fcp.attn_bwd_bias(q, k, v, self.kbuf, self.vbuf, bias, starts, out, lse, dout, self.dplan, shard, dq, dk, dv, dbias,
                          self.ws, scale=self.scale, zero_grads=zero_grads, stream=stream)
        return dq, dk, dv, dbias

    def backward(self, q, k, v, out, lse, dout, shard: int = -1, dq=None, dk=None, dv=None,
                 zero_kv_grads: bool = True, stream=None):
        with _on_stream(stream):
            if dq is None:
                dq = torch.empty(self.T, self.hq, self.d, dtype=torch.float32, device=self.device)
            if dk is None:
                dk = torch.zeros(self.T, self.hkv, self.d, dtype=torch.float32, device=self.device)
            elif zero_kv_grads:
                dk.zero_()
            if dv is None:
                dv = torch.zeros(self.T, self.hkv, self.d, dtype=torch.float32, device=self.device)
            elif zero_kv_grads:
                dv.zero_()
        fcp.attn_bwd(q, k, v, self.kbuf, self.vbuf, out, lse, dout, self.dplan, shard, dq, dk, dv,
                     self.ws, scale=self.scale, stream=stream)
        return dq, dk, dv

    def qk_norm_rope(self, q_in, k_in, v_in=None, wq=None, wk=None, inv_freq=None, norm: bool = True,
                     eps: float = 1e-6, interleaved: bool = False, shard: int = -1, q=None, k=None, v=None, stream=None):
        """Q, K (and V) for the attention from a layer's projection: every query
        and key head normed (weights wq, wk) and turned by its position inside
        its document (inv_freq; None: not turned). The inputs are [T][heads][d]
        tensors or slices of one fused tensor."""
        with _on_stream(stream):
            if q is None:
                q = torch.empty(self.T, self.hq, self.d, dtype=torch.bfloat16, device=self.device)
            if k is None:
                k = torch.empty(self.T, self.hkv, self.d, dtype=torch.bfloat16, device=self.device)
            if v is None and v_in is not None:
                v = torch.empty_like(k)
        fcp.qk_norm_rope(q_in, k_in, v_in, self.dplan, shard, q, k, v, wq=wq, wk=wk, inv_freq=inv_freq, norm=norm,
                         eps=eps, interleaved=interleaved, stream=stream)
        return q, k, v

    def qk_norm_rope_backward(self, dq, dk, dv, q_in, k_in, wq=None, wk=None, inv_freq=None, norm: bool = True,
                              eps: float = 1e-6, interleaved: bool = False, shard: int = -1, dq_in=None, dk_in=None,
                              dv_in=None, dwq=None, dwk=None, zero_grads: bool = False, stream=None):
        """Gradient of qk_norm_rope from backward()'s dq, dk and dv (None: no V):
        the bf16 gradients of its inputs, written into dq_in, dk_in and dv_in
        (slices of one fused gradient, for instance) or new tensors, and the fp32
        gradients of the weights, added to dwq and dwk where they are given
        (zero_grads: written there)."""
        def rows(heads):
            return torch.empty(self.T, heads, self.d, dtype=torch.bfloat16, device=self.device)
        with _on_stream(stream):
            dq_in = rows(self.hq) if dq_in is None else dq_in
            dk_in = rows(self.hkv) if dk_in is None else dk_in
            dv_in = rows(self.hkv) if dv_in is None and dv is not None else dv_in
            add = not zero_grads and (dwq is not None or dwk is not None)  # to the given ones: new ones start at zero
            make = torch.zeros if add else torch.empty
            if dwq is None and wq is not None:
                dwq = make(self.d, dtype=torch.float32, device=self.device)
            if dwk is None and wk is not None:
                dwk = make(self.d, dtype=torch.float32, device=self.device)
        fcp.qk_norm_rope_bwd(dq, dk, dv, q_in, k_in, self.dplan, shard, dq_in, dk_in, dv_in, dwq, dwk, self.ws, wq=wq,
                             wk=wk, inv_freq=inv_freq, norm=norm, eps=eps, interleaved=interleaved, add_dw=add,
                             stream=stream)
        return dq_in, dk_in, dv_in, dwq, dwk

    def residual_norm(self, x, y=None, gate=None, w_post=None, w_pre=None, post_norm: bool = True, pre_norm: bool = True,
                      gate_fn: str = "sigmoid", res_scale: float = 1.0, branch_scale: float = 1.0, eps: float = 1e-6,
                      shard: int = -1, x_out=None, h=None, stream=None):
        """The residual stream after a block and the next block's input, (x_out, h): the block's output
        y normed (post_norm), gated, scaled and added to the residual x, and that normed again (pre_norm;
        else h is None). x [T][n] bf16 or fp32, y and gate bf16; without y only the norm (x_out is then
        x itself where res_scale is 1 and it is not given)."""
        if h is not None and not pre_norm:
            raise ValueError("residual_norm: h is the norm's result: pre_norm = True with it")
        with _on_stream(stream):
            if x_out is None and (y is not None or res_scale != 1.0 or not pre_norm):
                x_out = torch.empty(x.shape, dtype=x.dtype, device=self.device)
            if h is None and pre_norm:
                h = torch.empty(x.shape, dtype=torch.bfloat16, device=self.device)
        fcp.residual_norm(x, y, gate, self.dplan, shard, x_out, h, w_post=w_post, w_pre=w_pre, post_norm=post_norm,
                          gate_fn=gate_fn, res_scale=res_scale, branch_scale=branch_scale, eps=eps, stream=stream)
        return x if x_out is None else x_out, h

    def residual_norm_backward(self, dh, dx_out, x_out, y=None, gate=None, w_post=None, w_pre=None, post_norm: bool = True,
                               gate_fn: str = "sigmoid", res_scale: float = 1.0, branch_scale: float = 1.0,
                               eps: float = 1e-6, shard: int = -1, dx=None, dy=None, dgate=None, dw_post=None, dw_pre=None,
                               zero_grads: bool = False, stream=None):
        """Gradient of residual_norm, (dx, dy, dgate, dw_post, dw_pre), from dh (None: no norm before the
        next block) and dx_out, the gradient along the residual (None: none). The fp32 gradients of the
        weights are added to dw_post and dw_pre where they are given (zero_grads: written there). Its
        workspace is made in the order of the call's stream."""
        like = x_out if x_out is not None else dx_out
        if like is None:
            raise ValueError("residual_norm_backward: x_out or dx_out is needed")
        n = like.shape[1]
        with _on_stream(stream):
            def rows(t, dtype):
                return torch.empty(t.shape, dtype=dtype, device=self.device)
            dx = rows(like, like.dtype) if dx is None else dx
            dy = rows(y, y.dtype) if dy is None and y is not None else dy
            dgate = rows(gate, gate.dtype) if dgate is None and gate is not None else dgate
            add = not zero_grads and (dw_post is not None or dw_pre is not None)  # to the given ones: new ones start at zero
            make = torch.zeros if add else torch.empty
            if dw_post is None and w_post is not None:
                dw_post = make(n, dtype=torch.float32, device=self.device)
            if dw_pre is None and w_pre is not None:
                dw_pre = make(n, dtype=torch.float32, device=self.device)
            ws = None
            if dw_post is not None or dw_pre is not None:
                ws = torch.empty(fcp.residual_norm_ws_bytes(n) // 4, dtype=torch.float32, device=self.device)
        fcp.residual_norm_bwd(dh, dx_out, x_out, y, gate, self.dplan, shard, dx, dy, dgate, dw_post, dw_pre, ws,
                              w_post=w_post, w_pre=w_pre, post_norm=post_norm, gate_fn=gate_fn, res_scale=res_scale,
                              branch_scale=branch_scale, eps=eps, add_dw=add, stream=stream)
        return dx, dy, dgate, dw_post, dw_pre

    def device_status(self) -> int:
        return fcp.device_status(self.ws)
