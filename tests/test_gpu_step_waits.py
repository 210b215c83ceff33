"""Bounded waits of the gated block's and Muon's products (failure detection without a fault), as tests/test_gpu_wait.py has
them for the GEMM: with a limit of 1 ns the first wait that is not already satisfied runs out, the single-CTA kernels record
XT_DEVERR_TIMEOUT, drain their copies and products, release their tensor memory and return; with the limit restored the same
call gives the same bits as before.  (A pair whose wait runs out may leave a copy of its odd CTA unwaited for, so the paired
kernels are left out, as the GEMM's is.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu

xt = pytest.importorskip("transformer_fwd_bwd_gb300.xt")


@pytest.fixture
def short_waits():
    xt.clear_device_errors()
    yield
    xt.set_wait_limit_ns(0)
    xt.gemm_set_pairing(0)
    xt.gemm_set_schedule(0)
    xt.clear_device_errors()


def runs_out_and_recovers(run):
    want = run()
    assert xt.device_errors() == 0
    xt.set_wait_limit_ns(1)
    run()
    assert xt.device_errors() & xt.XT_DEVERR_TIMEOUT
    xt.set_wait_limit_ns(0)
    xt.clear_device_errors()
    got = run()
    assert xt.device_errors() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_gated_block(short_waits):
    xt.gemm_set_pairing(1)
    xt.gemm_set_schedule(1)
    T, d, F = 700, 4096, 520
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.05).bfloat16()  # noqa: E731
    x, wu, wd, dy = n(T, d), n(d, 2 * F), n(F, d), n(T, d)

    def run():
        e = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        gu, h, dgu, dw = e(T, 2 * F), e(T, F), e(T, 2 * F), e(d, 2 * F)
        xt.xt_gated_mlp_fwd(x, wu, None, gu, h, None)
        xt.xt_gated_mlp_bwd(x, wu, wd, gu, h, dy, dgu, None, dw, None)
        torch.cuda.synchronize()
        return gu, h, dgu, dw
    runs_out_and_recovers(run)


def test_muon(short_waits):
    shapes = [(256, 2048), (100, 70)]
    g = torch.Generator(device="cuda").manual_seed(2)
    grads = [torch.randn(*s, generator=g, device="cuda") for s in shapes]

    def run():
        p, m = ([torch.zeros(*s, device="cuda") for s in shapes] for _ in range(2))
        xt.xt_muon_step(xt.muon_config(0.02), p, grads, m)
        torch.cuda.synchronize()
        return (*p, *m)
    runs_out_and_recovers(run)
