"""What log probabilities are by definition, kept by the rounded ones too: none above 0, no probability above 1 (a loss that takes
log(1 - p) or a root of -log p meets no NaN), and a row whose one token has all of the probability has neither an entropy
nor a gradient.

The sum of exponentials to the base of the largest is at least 1, whatever the exponential's error.  Where one token has it all,
logp = 0 and entropy = ln S, S - 1 within the exponential's 2 ulp (2⁻²²); the entropy's gradient p·(log p + H) is then a
difference of equal numbers, each rounded at most three times: 4·2⁻²⁴·2⁻²² ≤ 2⁻⁴⁰ of the upstream."""
import math

import pytest
import torch

from tests.test_gpu_token_logprobs import TD, forward

pytestmark = pytest.mark.gpu

xt = pytest.importorskip("transformer_fwd_bwd_gb300.xt")


# a warp's rows, a CTA's, a cluster's
@pytest.mark.parametrize("R,V", [(3000, 1), (2000, 7), (1000, 400), (700, 9001), (5, 50257)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_one_token_has_it_all(R, V, dtype, scale):
    g = torch.Generator(device="cuda").manual_seed(R + V)
    x = torch.full((R, V), -math.inf, device="cuda")
    tok = torch.randint(0, V, (R,), generator=g, device="cuda").int()
    rows = torch.arange(R, device="cuda")
    x[rows, tok.long()] = 30 * torch.randn(R, generator=g, device="cuda")
    x = x.to(TD[dtype])
    logp, H, stats, tl, ti = forward(x, tok, 1, scale)
    assert torch.equal(ti[:, 0], tok)
    assert (logp <= 0).all() and (tl <= 0).all() and (stats[:, 1] >= 0).all() and (H >= 0).all()
    assert (logp >= -2.0 ** -21).all() and (H <= 2.0 ** -21).all()
    dh = torch.randn(R, generator=g, device="cuda")
    dx = torch.empty(R, V, device="cuda")
    xt.xt_token_logprobs_bwd(x, tok, stats, H, None, dh, dx, scale=scale)
    assert (dx.abs() <= 2.0 ** -40 * dh.abs()[:, None]).all()


@pytest.mark.parametrize("R,V", [(3000, 60), (700, 9001), (5, 50257)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_none_above_nought(R, V, dtype):
    """Rows in which the largest logit stands far, further and furthest above the others."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(R, V, generator=g, device="cuda")
    rows = torch.arange(R, device="cuda")
    tok = torch.randint(0, V, (R,), generator=g, device="cuda").int()
    x[rows, tok.long()] = 12 + 40 * torch.rand(R, generator=g, device="cuda")
    x = x.to(TD[dtype])
    top = 5
    logp, H, stats, tl, ti = forward(x, tok, top)
    assert (logp <= 0).all() and (tl <= 0).all() and (stats[:, 1] >= 0).all() and (H >= 0).all()
    assert (tl[:, 1:] <= tl[:, :-1]).all() and torch.equal(ti[:, 0], tok) and torch.equal(tl[:, 0], logp)
