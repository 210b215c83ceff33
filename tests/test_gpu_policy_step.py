"""The operators of a training step's ends, middle and tail together, as a training program uses them: scaled embeddings,
gated feed-forward blocks, tied logits, the tokens' log probabilities and entropies as the loss, the gradients by the tape
against float64 autograd of the same formulas, then the Muon step on the blocks' matrices; and the block stack trained
with Muon.

Gradients go through bf16 matrix products, so they are held to the framework's tolerance of its GEMM paths,
‖g − r‖ ≤ 2e-2 ‖r‖ (tests/gpu_util.py)."""
import math

import numpy as np
import pytest
import torch

import synth
from tests.gpu_util import norm_err

pytestmark = pytest.mark.gpu

xt = pytest.importorskip("transformer_fwd_bwd_gb300.xt")
from transformer_fwd_bwd_gb300 import tape as T  # noqa: E402
from transformer_fwd_bwd_gb300.block import NativeBlock  # noqa: E402

BF = torch.bfloat16
ACTS = {0: torch.nn.functional.silu, 1: torch.nn.functional.gelu}


def model(V, d, F, layers, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, std: (std * torch.randn(*s, generator=g, device="cuda")).to(BF)  # noqa: E731
    return [r(V, d, std=0.5 * d ** -0.5)] + [t for _ in range(layers) for t in
                                             (r(d, 2 * F, std=d ** -0.5), r(F, d, std=F ** -0.5))]


def reference(params, ids, tokens, w, c, scale, act):
    leaves = [p.double().requires_grad_() for p in params]
    E = leaves[0]
    x = E[ids.long()] * math.sqrt(E.shape[1])
    for wu, wd in zip(leaves[1::2], leaves[2::2]):
        gate, up = (x @ wu).chunk(2, dim=1)
        x = x + (ACTS[act](gate) * up) @ wd
    lp = torch.log_softmax(scale * (x @ E.T), 1)
    loss = (w.double() * lp.gather(1, tokens.long()[:, None])[:, 0]).sum() + (c.double() * torch.special.entr(lp.exp()).sum(1)).sum()
    loss.backward()
    return float(loss.detach()), [t.grad for t in leaves]


@pytest.mark.parametrize("tokens,V,d,F,layers,act", [(300, 1000, 64, 136, 2, 0), (77, 520, 128, 264, 1, 1)])
def test_policy_loss_through_the_tape(tokens, V, d, F, layers, act):
    params = model(V, d, F, layers)
    g = torch.Generator(device="cuda").manual_seed(2)
    ids, tok = (torch.randint(0, V, (tokens,), generator=g, device="cuda").int() for _ in range(2))
    w, c = (torch.randn(tokens, generator=g, device="cuda") for _ in range(2))
    scale = 0.8
    want, grads = reference(params, ids, tok, w, c, scale, act)
    leaves = [T.leaf(p, grad_dtype=torch.float32) for p in params]
    x = T.embedding(leaves[0], ids, scale=math.sqrt(d))
    for wu, wd in zip(leaves[1::2], leaves[2::2]):
        x = T.add(x, T.gated_mlp(x, wu, wd, act))
    logp, H = T.token_logprobs(T.matmul(x, leaves[0], trans_b=True), tok, scale)
    loss = T.add(T.sum_all(T.mul(logp, T.leaf(w))), T.sum_all(T.mul(H, T.leaf(c))))
    # a sum of rounded terms that cancel: against the terms' magnitudes
    assert abs(float(loss.value) - want) <= 2e-2 * float((w.abs() * 8 + c.abs() * 8).sum())
    T.backward(loss)
    for leaf, r in zip(leaves, grads):
        assert leaf.grad.dtype == torch.float32
        assert norm_err(leaf.grad.cpu().numpy(), r.cpu().numpy()) <= 2e-2
    # the step on the blocks' matrices: new weights are their old ones plus the orthogonalised gradient's update
    mats = params[1:]
    masters, buf = [m.float() for m in mats], [torch.zeros(m.shape, device="cuda") for m in mats]
    old = [m.clone() for m in masters]
    xt.xt_muon_step(xt.muon_config(0.02), masters, [leaf.grad for leaf in leaves[1:]], buf, shadows=mats)
    for m, o, b, leaf, s in zip(masters, old, buf, leaves[1:], mats):
        up = (o - m).double() / (0.02 * 0.2 * math.sqrt(max(m.shape)))
        sv = torch.linalg.svdvals(up)
        assert torch.equal(b, leaf.grad) and torch.equal(s, m.to(BF))
        # the strong directions come out with singular values of 0.68 to 1.21 (float32 weights resolve 1e-3 of that)
        assert float(sv[0]) <= 1.21 + 1e-2 and float(sv[len(sv) // 4]) >= 0.68 - 1e-2
    assert xt.device_errors() == 0


def test_gated_weights_with_two_gradient_dtypes_and_a_shared_input():
    """x feeds two blocks; the weights' gradients are kept in different dtypes."""
    p = model(8, 64, 128, 2, seed=3)
    x0 = torch.randn(50, 64, device="cuda").to(BF)
    leaves = [t.double().requires_grad_() for t in [x0, *p[1:]]]
    out = sum((ACTS[0]((leaves[0] @ wu).chunk(2, 1)[0]) * (leaves[0] @ wu).chunk(2, 1)[1]) @ wd
              for wu, wd in zip(leaves[1::2], leaves[2::2]))
    out.sum().backward()
    ws = [T.leaf(t, grad_dtype=torch.float32 if i % 2 else BF) for i, t in enumerate(p[1:])]
    x = T.leaf(x0)
    y = T.add(T.gated_mlp(x, ws[0], ws[1]), T.gated_mlp(x, ws[2], ws[3]))
    T.backward(T.sum_all(y))
    for v, r in zip([x, *ws], leaves):
        assert norm_err(v.grad.float().cpu().numpy(), r.grad.cpu().numpy()) <= 2e-2


@pytest.mark.parametrize("dtype,bits", [("bf16", 32), ("f32", 32), ("bf16", 8)])
def test_block_stack_with_muon(dtype, bits):
    cfg = dict(synth.BLOCK_CONFIGS["tiny"], dtype=dtype)
    ids, tgt = (torch.from_numpy(a).cuda() for a in synth.block_tokens(cfg))
    blk = NativeBlock(cfg, device="cuda")
    blk.load(synth.block_params(cfg))
    blk.init_optimizer(lr=1e-3, state_bits=bits, matrices="muon")
    before = {k: v.clone() for k, v in blk.master.items()}
    blk.train_step([(ids, tgt), (ids, tgt)])
    mats = [k for k in blk.p if k.split(".")[-1] in ("Wqkv", "Wo", "Wup", "Wdown")]
    assert set(blk.momentum) == set(mats) and len(mats) == 4 * cfg["n_layers"]
    for k in mats:
        g = blk.g[k].double() * 0.5
        assert torch.equal(blk.momentum[k], blk.g[k] * 0.5)
        X = 1.95 * g
        X = X / (X.norm() + 1e-7)
        if X.shape[0] > X.shape[1]:
            X = X.T
        for _ in range(5):
            A = X @ X.T
            X = 3.4445 * X + (-4.7750 * A + 2.0315 * A @ A) @ X
        X = X.T if g.shape[0] > g.shape[1] else X
        want = before[k].double() * (1 - 0.02 * 0.1) - 0.02 * 0.2 * math.sqrt(max(g.shape)) * X
        assert float((blk.master[k].double() - want).norm()) <= 1e-5 * float(want.norm())
        assert torch.equal(blk.p[k], blk.master[k].to(blk.p[k].dtype))
    # the others step as they do beside AdamW on everything, but for the norm that clips them
    m, v = blk.moments()
    assert set(m) == set(v) == set(blk.p) - set(mats) and all(float(t.abs().max()) > 0 for t in m.values())
    assert np.isfinite(float(blk.grad_norm)) and xt.device_errors() == 0
    for _ in range(3):
        losses = blk.train_step([(ids, tgt)])
    assert all(np.isfinite(float(x)) for x in losses)
    with pytest.raises(ValueError):
        blk.init_optimizer(lr=1e-3, matrices="sgd")
