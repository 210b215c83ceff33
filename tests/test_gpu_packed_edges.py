"""Masked attention, rotary positions and the 8-bit AdamW step at their contracts' edges: values that are not finite in one
operand alone, scores that saturate their cap or overflow, plans of another batch, tiny epsilons, workspaces that
the binding allocates for another stream."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_util import empty
from tests.test_gpu_attention_masked import B8, Case, compare

pytestmark = pytest.mark.gpu

xt = pytest.importorskip("transformer_fwd_bwd_gb300.xt")

OUTPUTS = ("o", "lse", "dq", "dk", "dv")


def compare_tokens(got, val, tol, keep):
    """compare() over the tokens of `keep`."""
    at = lambda d: {n: d[n][:, keep] if n == "lse" else d[n][keep] for n in OUTPUTS}  # noqa: E731
    compare(at(got), at(val), at(tol))


@pytest.mark.parametrize("hd,Hkv,cap", [(64, 2, 0.0), (64, 1, 20.0), (128, 2, 20.0), (128, 1, 0.0)])
@pytest.mark.parametrize("which", ["q", "k", "v", "do"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_one_operand_of_a_token_is_not_finite(bad, which, hd, Hkv, cap):
    """The documents before and behind share tiles with the token's and are the definition's in every output: a key that
    is not finite leaves the other operands of the queries that see it finite, and their lse NaN."""
    c = Case(off=[0, 90, 200, 330], H=2, Hkv=Hkv, hd=hd, cap=cap)
    val, tol = c.reference()
    q, k, v = c.split(c.qkv)
    {"q": q, "k": k, "v": v, "do": c.do}[which][150] = bad
    keep = torch.ones(330, dtype=torch.bool, device="cuda")
    keep[90:200] = False
    compare_tokens(c.run(), val, tol, keep)


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("hd,Hkv", [(64, 2), (128, 1)])
def test_scores_that_overflow_stay_in_their_document(hd, Hkv, causal):
    """Finite queries and keys whose product leaves float32."""
    c = Case(off=[0, 90, 200, 330], H=2, Hkv=Hkv, hd=hd, causal=causal)
    val, tol = c.reference()
    q, k, _ = c.split(c.qkv)
    q[140] = 3e38
    k[150] = 3e38
    got = c.run()
    keep = torch.ones(330, dtype=torch.bool, device="cuda")
    keep[90:200] = False
    compare_tokens(got, val, tol, keep)
    assert not bool(torch.isfinite(got["lse"][:, 90:200]).all())


@pytest.mark.parametrize("H,Hkv", [(2, 2), (4, 1)], ids=["whole-groups", "split-group"])
def test_plan_of_another_length_leaves_gradients_alone(H, Hkv):
    """With a group of query heads in parts the parts' join writes nothing either."""
    c = Case(off=[0, 300], H=H, Hkv=Hkv)
    q, k, v = c.split(c.qkv)
    got = c.run()
    plan = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    xt.xt_attention_plan(plan, 260, 1)
    d = [empty((300, n * 64), "bf16", fill=3.0) for n in (H, Hkv, Hkv)]
    xt.xt_attention_masked_bwd(q, k, v, got["o"], c.do, got["lse"], *d, plan, H, Hkv, 64)
    try:
        assert xt.device_errors() == xt.XT_DEVERR_PLAN
        assert all(bool((t == 3.0).all()) for t in d)
    finally:
        xt.clear_device_errors()
