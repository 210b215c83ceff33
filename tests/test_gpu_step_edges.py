"""What a training step's operators (sorted embeddings, the gated block, Muon) have to hold beside their ordinary calls: plans
made while other kernels hold the SMs, the override that keeps paired kernels
out, workspaces made for larger batches."""
import re

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


def captured(fn, path):
    """A graph of what fn launches, as the driver prints it (kernels by name)."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph):
        fn()
    graph.debug_dump(str(path))
    return path.read_text()


@pytest.mark.filterwarnings("ignore:DEBUG")
def test_muon_without_pairs(tmp_path):
    """xt_gemm_set_pairing(1), never a paired kernel, holds for Muon's products too, and X is as accurate."""
    shapes = [(300, 700)] * 14 + [(769, 264)] * 8 + [(256, 256)] * 5   # tiles for pairs
    g = torch.Generator(device="cuda").manual_seed(4)
    grads = [torch.randn(*s, generator=g, device="cuda") for s in shapes]

    def run():
        p, m = ([torch.zeros(*s, device="cuda") for s in shapes] for _ in range(2))
        xt.xt_muon_step(xt.muon_config(0.02), p, grads, m)
        return p
    with_pairs = run()
    pair, one = (re.compile(rf"muon_product_kernel(?:<{k}>|ILi{k}E)") for k in (2, 1))
    assert pair.search(captured(run, tmp_path / "pairs.dot"))
    try:
        xt.gemm_set_pairing(1)
        single = run()
        text = captured(run, tmp_path / "single.dot")
    finally:
        xt.gemm_set_pairing(0)
    assert one.search(text) and not pair.search(text)
    # both are within 9e-4 of the formula's X (tests/test_gpu_muon.py), whose norm is at least 0.68 of its root rank
    for a, b in zip(with_pairs, single):
        assert float((a - b).norm()) <= 2 * 9e-4 * float(a.norm())


def test_embedding_workspace_of_a_larger_batch():
    """A batch just short of the length at which its pieces grow longer needs more room than the longer ones."""
    V, d = 1000, 768
    g = torch.Generator(device="cuda").manual_seed(5)
    ws = xt.embedding_sorted_workspace(52000, d)
    for T in (51800, 25900, 3):
        ids = torch.randint(0, V, (T,), generator=g, device="cuda").int()
        dh = torch.randn(T, d, generator=g, device="cuda")
        plan = xt.embedding_plan_buffer(T)
        xt.xt_embedding_plan(ids, V, plan)
        dE, own = torch.empty(V, d, device="cuda"), torch.empty(V, d, device="cuda")
        xt.xt_embedding_sorted_bwd(plan, dh, dE, ws=ws)
        xt.xt_embedding_sorted_bwd(plan, dh, own)
        assert torch.equal(dE, own)
        want = torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, ids.long(), dh.double())
        mag = torch.zeros_like(want).index_add_(0, ids.long(), dh.double().abs())
        # at most 32 additions in a piece, then the pieces of an id
        count = int(torch.bincount(ids).max())
        assert ((dE.double() - want).abs() <= (count + 2) * 2.0 ** -24 * mag).all()
