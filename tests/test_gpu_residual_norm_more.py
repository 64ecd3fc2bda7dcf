"""The residual norm on the GPU, more of it: fp32 rows too wide for the forward's ring in shared memory (more than 14336
values), in every form of the call."""
import pytest
import torch

from test_gpu_residual_norm import KW, check, forward_reference, make, run_forward, session, within

pytestmark = pytest.mark.gpu

WIDE = [14328, 14336, 14344, 15000, 16384]  # on both sides of the switch


@pytest.mark.parametrize("n", WIDE)
@pytest.mark.parametrize("gate", ["sigmoid", "plain", None])
@pytest.mark.parametrize("post_norm", [True, False])
def test_widest_fp32_rows(cuda, n, gate, post_norm):
    w = {14344: torch.bfloat16, 15000: None}.get(n, torch.float32)
    x = make(90, n, seed=n, gate=gate, res=torch.float32, w=w)
    check(session([50, 40]), x, dict(KW, post_norm=post_norm, gate_fn=gate or "plain"))


@pytest.mark.parametrize("n", WIDE[1:])
def test_widest_fp32_rows_without_a_block(cuda, n):
    x = make(200, n, seed=n, block=False, res=torch.float32)
    s = session([200])
    for kw in (dict(KW, res_scale=1.0), KW):
        x_out, h = run_forward(s, x, kw)
        want = forward_reference(x, kw)
        within(h, want["h"], "h")
        within(x_out, want["x_out"], "x_out")


@pytest.mark.parametrize("n", WIDE[1:4])
def test_widest_fp32_rows_of_shards_in_place(cuda, n):
    """Shard by shard, the residual in place, more rows than CTAs; the other shards' rows stay as they were."""
    docs, cp = [300, 1, 250, 49], 2
    s = session(docs, cp, "wholedoc")
    x = make(sum(docs), n, seed=n, res=torch.float32)
    want = forward_reference(x, KW)
    residual, h = x["x"].clone(), torch.full((sum(docs), n), torch.nan, dtype=torch.bfloat16, device="cuda")
    done = torch.zeros(sum(docs), dtype=torch.bool, device="cuda")
    for j in range(cp):
        run_forward(s, dict(x, x=residual), KW, shard=j, x_out=residual, h=h)
        done[torch.from_numpy(s.plan.query_indices(j)).cuda().long()] = True
        assert torch.equal(residual[~done], x["x"][~done]) and torch.equal(h.isnan().all(1), ~done)
    within(residual, want["x_out"], "x_out")
    within(h, want["h"], "h")
