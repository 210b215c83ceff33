"""What a training step's operators (sorted embeddings, the gated block, Muon) have to hold beside their ordinary calls: plans
made while other kernels hold the SMs."""
import pytest
import torch

pytestmark = pytest.mark.gpu

xt = pytest.importorskip("transformer_fwd_bwd_gb300.xt")


def entries(plan, T):
    """(ids, tokens) of a plan's sorted entries."""
    e = plan[16:16 + 8 * T].view(torch.int64)
    return e >> 32, e & 0xFFFFFFFF


def test_plans_beside_kernels_that_hold_the_gpu():
    """Clusters of 4, 8 and 16 CTAs on their own streams while matrix products fill the SMs, so that a cluster's CTAs start at
    different times: every plan is the ids' stable order."""
    V = 50304
    g = torch.Generator(device="cuda").manual_seed(3)
    sets = [torch.randint(0, V, (T,), generator=g, device="cuda").int() for T in (2049, 3000, 8191, 16384, 70001)]
    plans = [xt.embedding_plan_buffer(ids.numel()) for ids in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    a = torch.randn(4096, 4096, device="cuda").bfloat16()
    torch.cuda.synchronize()
    for _ in range(10):
        for _ in range(3):
            a @ a
        for plan in plans:
            plan.fill_(255)
        torch.cuda.current_stream().synchronize()
        for _ in range(3):
            a @ a
        for ids, plan, st in zip(sets, plans, streams):
            xt.xt_embedding_plan(ids, V, plan, s=st)
        torch.cuda.synchronize()
        for ids, plan in zip(sets, plans):
            want = torch.sort(ids.long(), stable=True)
            got, at = entries(plan, ids.numel())
            assert torch.equal(got, want.values) and torch.equal(at, want.indices)
    assert xt.device_errors() == 0
