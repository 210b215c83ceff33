"""Bounded waits of the paired-CTA products (failure detection without a fault), as tests/test_gpu_wait.py has them for the
single-CTA ones: with a limit of 1 ns the first wait that is not already satisfied runs out in either CTA, at different fills
of their stages.  The kernels record XT_DEVERR_TIMEOUT, wait for every copy that any CTA of the cluster asked for, release
their tensor memory and return at once (a copy that were waited for in vain would take the two seconds of that wait's own
limit); with the limit restored the same call gives the same bits as before."""
import time

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


def runs_out_and_recovers(run, repeats=3):
    want = run()
    assert xt.device_errors() == 0
    for _ in range(repeats):
        xt.set_wait_limit_ns(1)
        t0 = time.perf_counter()
        run()
        assert time.perf_counter() - t0 < 1.0
        assert xt.device_errors() & xt.XT_DEVERR_TIMEOUT
        xt.set_wait_limit_ns(0)
        xt.clear_device_errors()
        got = run()
        assert xt.device_errors() == 0
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def runs_out_somewhere(run, limits=(200, 500, 1000, 2000, 4000, 8000)):
    """Limits within which some waits end and others do not: the CTAs stop at fills of their own in the middle of the work."""
    want = run()
    for limit in limits:
        xt.set_wait_limit_ns(limit)
        t0 = time.perf_counter()
        got = run()
        assert time.perf_counter() - t0 < 1.0
        if xt.device_errors() == 0:
            assert all(torch.equal(a, b) for a, b in zip(want, got))
        xt.set_wait_limit_ns(0)
        xt.clear_device_errors()
        got = run()
        assert xt.device_errors() == 0
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def kinds(fn):
    """Tile-width code of every product that fn launches: 1000 and more are pairs'."""
    xt.profile_gemm(16)
    try:
        fn()
        torch.cuda.synchronize()
        return [int(r[4]) for r in xt.profile_gemm_read(shapes=True)[2]]
    finally:
        xt.profile_gemm(0)


@pytest.mark.parametrize("pairing", [2, 3])  # pairs; two pairs that multicast to each other
def test_gemm(pairing, short_waits):
    xt.gemm_set_pairing(pairing)
    xt.gemm_set_schedule(1)
    M, N, K = 1024, 1024, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    A, B = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((M, K), (K, N)))
    desc = xt.matmul_desc(M, N, K)

    def run():
        C = torch.zeros(M, N, device="cuda")
        xt.xt_matmul_fwd(desc, A, B, C)
        torch.cuda.synchronize()
        return [C]
    codes = kinds(run)
    assert len(codes) == 1 and codes[0] >= 1000
    runs_out_and_recovers(run)
    runs_out_somewhere(run)


def test_gated_block(short_waits):
    T, d, F = 4097, 1024, 2056
    g = torch.Generator(device="cuda").manual_seed(2)
    n = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.05).bfloat16()  # noqa: E731
    x, wu, wd, dy = n(T, d), n(d, 2 * F), n(F, d), n(T, d)
    xt.gemm_set_schedule(1)

    def run():
        e = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        gu, h, dgu, dw = e(T, 2 * F), e(T, F), e(T, 2 * F), e(d, 2 * F)
        xt.xt_gated_mlp_fwd(x, wu, None, gu, h, None)
        xt.xt_gated_mlp_bwd(x, wu, wd, gu, h, dy, dgu, None, dw, None)
        torch.cuda.synchronize()
        return gu, h, dgu, dw
    assert kinds(run)[:2] == [1256, 1256]
    runs_out_and_recovers(run)
    runs_out_somewhere(run)


def test_muon(short_waits):
    """Enough matrices for the tiles that pairs share."""
    shapes = [(300, 700)] * 14 + [(769, 264)] * 8 + [(256, 256)] * 5
    g = torch.Generator(device="cuda").manual_seed(3)
    grads = [torch.randn(*s, generator=g, device="cuda") for s in shapes]

    def run():
        p, m = ([torch.zeros(*s, device="cuda") for s in shapes] for _ in range(2))
        xt.xt_muon_step(xt.muon_config(0.02), p, grads, m)
        torch.cuda.synchronize()
        return (*p, *m)
    runs_out_and_recovers(run)
    runs_out_somewhere(run)
