"""Windowed attention on the GPU, more of it: gradients from a bf16 output, scales, groups of many sizes, shard by shard
with sinks that a shard holds a part of, gradients added to given ones."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import window as W
from test_gpu_window import BF16, NAMES, make, session, step, within
from test_gpu_window import reference as full_reference

pytestmark = pytest.mark.gpu


def reference(q, k, v, do, docs, window, sinks, scale=None):
    """Results and bounds; dV's with what dO's fp16 copies lose besides: a row i is divided by a power of two of at most
    |dO_i|, so an element below fp16's normal range is off by 2^-25 |dO_i|, times a probability of at most 1, over the
    queries (and heads of the group) that see a key."""
    want = full_reference(q, k, v, do, docs, window, sinks, scale)
    queries = q.shape[1] // k.shape[1] * (max(docs) if sinks else min(window, max(docs)))
    ref, err = want["dv"]
    return dict(want, dv=(ref, err + queries * 2.0 ** -25 * float(do.float().norm(dim=-1).max())))



def of_rounded_output(x, want, docs, window, sinks):
    """The bounds of dQ and dK where D = <dO, O> takes O rounded to bf16: O is off by half a step, 2^-8 |O|, more (and by as
    much of its own error), which P carries into dS and the factors K and Q on. (1.01: the fp16 roundings of that part.)"""
    q, k, v, do = (A.to_f64(t) for t in x)
    G, scale = q.shape[1] // k.shape[1], 1 / math.sqrt(q.shape[2])
    dq, dk = want["dq"][1].copy(), want["dk"][1].copy()
    a = 0
    for n in docs:
        e = a + n
        seen = W.visible(n, window, sinks)
        for h in range(q.shape[1]):
            s = np.where(seen, scale * q[a:e, h] @ k[a:e, h // G].T, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            O, eO = (t[a:e, h] for t in want["out"])
            off = 1.01 * p * (np.abs(do[a:e, h]) * BF16 * (np.abs(O) + eO)).sum(1, keepdims=True)
            dq[a:e, h] += scale * off @ np.abs(k[a:e, h // G])
            dk[a:e, h // G] += scale * off.T @ np.abs(q[a:e, h])
        a = e
    return dict(want, dq=(want["dq"][0], dq), dk=(want["dk"][0], dk))


@pytest.mark.parametrize("docs,cp,hq,hkv,d,window,sinks", [
    ([1, 300, 129, 600], 2, 4, 2, 128, 100, 4), ([700], 4, 5, 5, 64, 64, 20), ([500, 37], 1, 3, 1, 64, 257, 0)])
def test_gradients_from_a_bf16_output(cuda, docs, cp, hq, hkv, d, window, sinks):
    x = make(docs, hq, hkv, d, seed=21)
    s = session(docs, cp, "perdoc", hq, hkv, d, window, sinks)
    q, k, v, do = (t.cuda() for t in x)
    s.gather(k, v)
    out, lse = s.forward(q, k, v)
    assert out.dtype == torch.bfloat16
    want = of_rounded_output(x, reference(*x, docs, window, sinks), docs, window, sinks)
    within(out.cpu(), want, "out", extra=BF16)
    for name, y in zip(NAMES[2:], s.backward(q, k, v, out, lse, do)):
        within(y.cpu(), want, name)
    assert s.device_status() == 0


@pytest.mark.parametrize("scale", [0.02, 0.3])
def test_scales(cuda, scale):
    docs, hq, hkv, d, window, sinks = [400, 90], 4, 2, 64, 77, 3
    x = make(docs, hq, hkv, d, seed=22)
    s = session(docs, 2, "perdoc", hq, hkv, d, window, sinks, scale=scale)
    want = reference(*x, docs, window, sinks, scale=scale)
    for name, y in zip(NAMES, step(s, [t.cuda() for t in x])):
        within(y.cpu(), want, name)


@pytest.mark.parametrize("policy", ["llama3", "perdoc", "wholedoc", "hybrid", "hybrid_tiles"])
@pytest.mark.parametrize("hq,hkv,d", [(7, 1, 64), (9, 3, 128), (1, 1, 128), (10, 2, 64)])
def test_groups_and_policies(cuda, policy, hq, hkv, d):
    docs, cp, window, sinks = [3, 260, 1, 500, 90, 170], 4, 45, 12
    x = make(docs, hq, hkv, d, seed=hq)
    s = session(docs, cp, policy, hq, hkv, d, window, sinks)
    want = reference(*x, docs, window, sinks)
    for name, y in zip(NAMES, step(s, [t.cuda() for t in x])):
        within(y.cpu(), want, name)


@pytest.mark.parametrize("hq,hkv", [(3, 1), (4, 4), (4, 2)])
def test_shards_that_hold_a_part_of_the_sinks(cuda, hq, hkv):
    """The sinks are received as one run, own ones among them; dK and dV are added to what is there."""
    docs, cp, d, window, sinks = [9, 20, 31, 40, 150], 4, 64, 3, 37
    x = make(docs, hq, hkv, d, seed=23)
    want = reference(*x, docs, window, sinks)
    s = session(docs, cp, "perdoc", hq, hkv, d, window, sinks)
    q, k, v, do = (t.cuda() for t in x)
    T = sum(docs)
    out, lse = torch.empty(T, hq, d, device="cuda"), torch.empty(hq, T, device="cuda")
    dq = torch.empty(T, hq, d, device="cuda")
    dk, dv = (torch.full((T, hkv, d), 3.0, device="cuda") for _ in range(2))
    for j in range(cp):
        s.gather(k, v, shard=j)
        s.forward(q, k, v, shard=j, out=out, lse=lse)
        s.backward(q, k, v, out, lse, do, shard=j, dq=dq, dk=dk, dv=dv, zero_kv_grads=False)
    assert s.device_status() == 0
    for name, y in zip(NAMES, (out, lse, dq, dk - 3, dv - 3)):
        ref, err = want[name]
        # At most 16 reduce-adds to a row (a unit of each of its document's 8 pieces for its sinks, those whose windows hold
        # it) and the difference, each rounded at a value of at most 3 and the sum of the gradient's terms, of which err is
        # 2^-11 and more.
        more = 17 * 2.0 ** -24 * (3 + 2048 * err) if name in ("dk", "dv") else 0
        within(y.cpu(), {name: (ref, err + more)}, name)
