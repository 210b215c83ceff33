"""Muon over gradients of any finite size, against its formulas in 64 bits: entries whose squares lie outside float32's range on
either side, or whose norm itself does.

Tolerances as in tests/test_gpu_muon.py: X within sqrt(15)·a⁵·2⁻²¹ = 9e-4 of the formula's in norm, and three float32
roundings of the weights."""
import math

import pytest
import torch

from tests.test_gpu_muon import ABC, EPS, X_TOL

pytestmark = pytest.mark.gpu

xt = pytest.importorskip("transformer_fwd_bwd_gb300.xt")


def orthogonalised(U, eps, steps=5):
    X = U / (U.norm() + eps)
    X = X.T if U.shape[0] > U.shape[1] else X
    for _ in range(steps):
        A = X @ X.T
        X = ABC[0] * X + (ABC[1] * A + ABC[2] * (A @ A)) @ X
    return X.T if U.shape[0] > U.shape[1] else X


def check(grads, eps, momentum=0.5, nesterov=1):
    shapes = [tuple(g.shape) for g in grads]
    gen = torch.Generator(device="cuda").manual_seed(9)
    P = [0.02 * torch.randn(*s, generator=gen, device="cuda") for s in shapes]
    old, M = [p.clone() for p in P], [torch.zeros(s, device="cuda") for s in shapes]
    xt.xt_muon_step(xt.muon_config(0.02, momentum=momentum, eps=eps, nesterov=nesterov), P, grads, M)
    for p, o, g, m, s in zip(P, old, grads, M, shapes):
        assert torch.equal(m, g)
        U = g.double() * (1 + momentum * nesterov)
        X = orthogonalised(U, float(torch.tensor(eps, dtype=torch.float32)))
        up = 0.02 * 0.2 * math.sqrt(max(s))
        want = o.double() - up * X
        assert float((p.double() - want).norm()) <= up * X_TOL + 3 * EPS * float(want.norm() + up * X.norm())
    assert xt.device_errors() == 0


# squares beyond float32 at either end; the last two: the norm of 3e6 entries of 1e38 is beyond it too, and entries of 1e-38
# need a factor that is
@pytest.mark.parametrize("size,eps", [(1e18, 1e-7), (1e19, 1e-7), (1e25, 1e-7), (1e30, 1e-30), (1e-18, 1e-30), (1e-22, 1e-30),
                                      (1e-25, 1e-35), (1e-30, 1e-38), (1e-25, 1e-7), (3e37, 1e-7), (1e-37, 1e-40)])
def test_sizes(size, eps):
    gen = torch.Generator(device="cuda").manual_seed(1)
    mk = lambda r, c: size * torch.randn(r, 6, generator=gen, device="cuda").clamp(-2, 2) @ \
        torch.eye(6, c, device="cuda") + 0.2 * size * torch.randn(r, c, generator=gen, device="cuda").clamp(-2, 2)  # noqa: E731
    check([mk(64, 200), mk(200, 64), mk(130, 130)], eps)


def test_a_norm_beyond_float32():
    gen = torch.Generator(device="cuda").manual_seed(2)
    g = (torch.randn(1024, 3000, generator=gen, device="cuda").clamp(-2, 2) / 2) * 2e38
    check([g], 1e-7, momentum=0.0, nesterov=0)


def test_one_large_entry_among_small_ones():
    """The squares of one piece of the sum leave the range, those of the others do not."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    g = 1e-3 * torch.randn(300, 500, generator=gen, device="cuda")
    big = g.clone()
    big[7, 11] = 1e21
    tiny = torch.zeros_like(g)
    tiny[:3] = 1e-24 * torch.randn(3, 500, generator=gen, device="cuda")
    check([g, big, tiny], 1e-30)
