"""The gated feed-forward block, element by element: every product against the same product in 64 bits of the very operands
that it reads (h, g and u, dg and du as the block stored them), so that a bound holds one rounding and the float32 sums alone
and no wrong element hides in a norm.

Tolerances: a rounding to bf16 is off by at most 2⁻⁸ of the value, to float32 by 2⁻²⁴; a float32 sum of K products by (K + 2)·2⁻²⁴
of their magnitudes (plus 4 more additions where it is made in parts).  act and act' in float32: the exponential of an argument
t is off by at most (|t| + 4)·2⁻²², the quotient and the products by a few 2⁻²⁴; together (t + 16)·2⁻²² of the values that are
combined, |g| and 1 at most, with t = |g| for silu and g²/2 for gelu, and 2⁻²⁰ of them for gelu's polynomial."""
import pytest
import torch

from tests.test_gpu_gated_mlp import CASES, HALF, act64, bufs, make

pytestmark = pytest.mark.gpu

xt = pytest.importorskip("transformer_fwd_bwd_gb300.xt")

EPS = 2.0 ** -24


def product(a, b):
    """a b in 64 bits and the bound of its float32 sum."""
    a, b = a.double(), b.double()
    return a @ b, (a.shape[1] + 6) * EPS * (a.abs() @ b.abs())


def held(got, want, tol, what):
    half = HALF if got.dtype == torch.bfloat16 else EPS
    bound = half * (want.abs() + tol) + tol + 1e-38
    worst = float(((got.double() - want).abs() / bound).max()) if want.numel() else 0.0
    assert worst <= 1.0, (what, worst)


@pytest.mark.parametrize("T,d,F,act,grad", CASES + [(700, 768, 2048, 1, "f32"), (1, 2048, 5464, 0, "f32"),
                                                    (257, 2048, 5464, 1, "bf16")])
def test_every_element(T, d, F, act, grad):
    x, wu, wd, dy = make(T, d, F, 7)
    o = bufs(T, d, F, grad)
    ws = xt.gated_mlp_workspace(T, d, F)
    xt.xt_gated_mlp_fwd(x, wu, wd, o["gu"], o["h"], o["y"], act=act, ws=ws)
    xt.xt_gated_mlp_bwd(x, wu, wd, o["gu"], o["h"], dy, o["dgu"], o["dx"], o["dw_up"], o["dw_down"], act=act, ws=ws)
    # h from the float32 projections
    gu, e = product(x, wu)
    held(o["gu"], gu, e, "gu")
    (g, u), (eg, eu) = gu.split(F, 1), e.split(F, 1)
    a, _ = act64(g, act)
    slack = ((g.abs() if act == 0 else g * g / 2) + 16) * 2.0 ** -22 + (2.0 ** -20 if act else 0.0)
    ea = slack * g.abs() + 1.2 * eg  # the activations' slopes are at most 1.2
    held(o["h"], a * u, ea * u.abs() + a.abs() * eu + ea * eu + 4 * EPS * (a * u).abs(), "h")
    held(o["y"], *product(o["h"], wd), "y")
    # dg and du from the stored projections
    g, u = (t.double() for t in o["gu"].split(F, 1))
    a, da = act64(g, act)
    slack = ((g.abs() if act == 0 else g * g / 2) + 16) * 2.0 ** -22 + (2.0 ** -20 if act else 0.0)
    dh, edh = product(dy, wd.T)
    eda = slack * (1 + g.abs())
    dg, du = dh * u * da, dh * a
    held(o["dgu"][:, :F], dg, u.abs() * (dh.abs() * eda + edh * (da.abs() + eda)) + 4 * EPS * dg.abs(), "dg")
    held(o["dgu"][:, F:], du, dh.abs() * slack * g.abs() + edh * (a.abs() + slack * g.abs()) + 4 * EPS * du.abs(), "du")
    held(o["dx"], *product(o["dgu"], wu.T), "dx")
    held(o["dw_up"], *product(x.T, o["dgu"]), "dw_up")
    held(o["dw_down"], *product(o["h"].T, dy), "dw_down")
    assert xt.device_errors() == 0
