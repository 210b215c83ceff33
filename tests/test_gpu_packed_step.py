"""The packed-document operators together, as a training program uses them: an attention layer on rows that hold
several documents (rotary positions over several axes on q and k, masked attention, output projection) through
the tape, its gradients against float64 autograd of the same formulas, and the 8-bit AdamW step on them; the
block stack trained with 8-bit state; two layers of one plan at once on two streams; waits that run out.

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


def layer_data(tokens, d, H, Hkv, hd, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, std=1.0: (std * torch.randn(*s, generator=g, device="cuda")).to(BF)  # noqa: E731
    return (r(tokens, d), r(d, H * hd, std=d ** -0.5), r(d, Hkv * hd, std=d ** -0.5), r(d, Hkv * hd, std=d ** -0.5),
            r(H * hd, d, std=(H * hd) ** -0.5), r(tokens, d))


def reference(x, wq, wk, wv, wo, w, pos, sections, off, prefix, H, Hkv, hd, cap, slopes):
    """Gradients of Σ w∘(attention layer of x) by autograd in float64."""
    leaves = [t.double().requires_grad_() for t in (x, wq, wk, wv, wo)]
    x, wq, wk, wv, wo = leaves
    i, th = 0, []
    for a, n in enumerate(sections):
        for _ in range(n):
            th.append(pos[a].double() * 10000.0 ** (-2.0 * i / hd))
            i += 1
    th = torch.stack(th, 1)[:, None]

    def rot(t, heads):
        t = t.view(-1, heads, hd)
        a, b = t[..., :hd // 2], t[..., hd // 2:]
        return torch.cat([a * th.cos() - b * th.sin(), b * th.cos() + a * th.sin()], -1)
    q, k, v = rot(x @ wq, H), rot(x @ wk, Hkv), (x @ wv).view(-1, Hkv, hd)
    outs = []
    for d in range(len(off) - 1):
        at = slice(off[d], off[d + 1])
        m = off[d + 1] - off[d]
        j = torch.arange(m, device="cuda")
        see = (j[None, :] <= j[:, None]) | (j < prefix[d])[None, :]
        heads = []
        for h in range(H):
            s = q[at, h] @ k[at, h // (H // Hkv)].T / math.sqrt(hd)
            s = cap * torch.tanh(s / cap) - float(slopes[h]) * (j[:, None] - j[None, :]).abs()
            heads.append(torch.softmax(s.masked_fill(~see, -math.inf), -1) @ v[at, h // (H // Hkv)])
        outs.append(torch.cat(heads, 1))
    loss = ((torch.cat(outs) @ wo) * w.double()).sum()
    loss.backward()
    return [t.grad for t in leaves]


@pytest.mark.parametrize("hd", [64, 128])
def test_packed_layer_gradients_and_8_bit_step(hd):
    tokens, d, H, Hkv, cap = 420, 256, 4, 2, 20.0
    off, prefix = [0, 130, 131, 420], [40, 0, 100]
    sections = [hd // 8, hd // 4, hd // 8]
    data = layer_data(tokens, d, H, Hkv, hd, 1)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pos = torch.stack([torch.cat([torch.arange(off[k + 1] - off[k]) * (a + 1) for k in range(3)]) for a in range(3)])
    pos = pos.to(torch.int32).cuda()
    slopes = torch.exp2(-2.0 * torch.arange(1, H + 1, device="cuda").float())
    plan = xt.attention_plan_buffer(tokens)
    xt.xt_attention_plan(plan, tokens, 3, ints(off), None, ints(prefix))
    x, wq, wk, wv, wo = (T.leaf(t, grad_dtype=torch.float32) for t in data[:5])
    q = T.rope_axes(T.matmul(x, wq), pos, sections, H, hd)
    k = T.rope_axes(T.matmul(x, wk), pos, sections, Hkv, hd)
    o = T.attention_masked(q, k, T.matmul(x, wv), plan, H, Hkv, hd, cap=cap, slopes=slopes)
    T.backward(T.sum_all(T.mul(T.matmul(o, wo), T.leaf(data[5]))))
    torch.cuda.synchronize()
    assert xt.device_errors() == 0
    want = reference(*data, pos, sections, off, prefix, H, Hkv, hd, cap, slopes)
    for name, leaf, r in zip(("x", "wq", "wk", "wv", "wo"), (x, wq, wk, wv, wo), want):
        assert norm_err(leaf.grad.double().cpu().numpy(), r.cpu().numpy()) <= 2e-2, name
    # the step: float32 master weights, state in 8 bits, bf16 working copies rewritten
    params = [t.value.float().view(-1) for t in (wq, wk, wv, wo)]
    grads = [t.grad.view(-1) for t in (wq, wk, wv, wo)]
    state = xt.adamw8_state(params)
    before = [p.clone() for p in params]
    shadows = [torch.empty_like(t.value) for t in (wq, wk, wv, wo)]
    norm = torch.zeros(1, device="cuda")
    xt.xt_adamw8_step(xt.adamw_config(1e-2, eps=1e-8, weight_decay=0.1, max_grad_norm=1.0), params, grads, *state,
                      shadows=[s.view(-1) for s in shadows], norm_out=norm)
    total = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    assert abs(float(norm) - total) <= 1e-6 * total
    for p, b, g, s in zip(params, before, grads, shadows):
        # the first step: m̂ = g', v̂ = g'², so the update is lr·g'/(|g'| + ε)
        gc = g.double() * min(1.0, 1.0 / (total + 1e-6))
        ref = b.double() * (1 - 1e-3) - 1e-2 * gc / (gc.abs() + 1e-8)
        assert float((p.double() - ref).abs().max()) <= 1e-2 * 32 * 2.0 ** -24 + 4 * 2.0 ** -24 * float(b.abs().max())
        assert torch.equal(s.view(-1), p.to(BF))


def test_block_stack_with_8_bit_state():
    """The stack's train_step with 8-bit moments: the first step equals the 32-bit one's to the rounding of the two
    formulas, and the state reads back as moments."""
    cfg = dict(synth.BLOCK_CONFIGS["gpt12"], B=1, S=64, d=64, H=1, hd=64, F=128, V=256, n_layers=1)
    ids, tgt = (torch.from_numpy(a).cuda() for a in synth.block_tokens(cfg))
    masters = []
    for bits in (32, 8):
        nb = NativeBlock(cfg, device="cuda:0", training=True)
        nb.load(synth.block_params(cfg))
        nb.init_optimizer(lr=1e-3, state_bits=bits)
        losses = nb.train_step([(ids, tgt)])
        m, v = nb.moments()
        torch.cuda.synchronize()
        assert math.isfinite(float(losses[0]))
        masters.append((nb, {k: t.clone() for k, t in nb.master.items()}, m, v))
        assert all(torch.equal(nb.p[k], nb.master[k].to(nb.p[k].dtype)) for k in nb.p)
    (a, pa, ma, va), (b, pb, mb, vb) = masters
    for k in pa:
        # lr times the difference of two float32 evaluations of m̂/(√v̂ + ε), the gradient equal bit for bit
        assert float((pa[k] - pb[k]).abs().max()) <= 1e-3 * 64 * 2.0 ** -24 + 2.0 ** -23 * float(pa[k].abs().max()), k
        # codes: (c ± ½)² about c² of the block's largest: at most 1/127 of the largest for m
        assert float((ma[k] - mb[k]).abs().max()) <= float(ma[k].abs().max()) * (1.0 / 127 + 1e-5), k
        assert float((va[k] - vb[k]).abs().max()) <= float(va[k].abs().max()) * (2.0 / 127 + 1e-5), k
    with pytest.raises(ValueError):
        b.init_optimizer(lr=1e-3, state_bits=16)
    for _ in range(2):   # later steps run on the decoded state
        b.train_step([(ids, tgt)])
    torch.cuda.synchronize()
    assert all(bool(torch.isfinite(t).all()) for t in b.master.values())


def attention_run(seed, plan, tokens, H, hd, stream=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(tokens, 3 * H * hd, generator=g, device="cuda").to(BF)
    do = torch.randn(tokens, H * hd, generator=g, device="cuda").to(BF)
    out = [torch.zeros(tokens, H * hd, device="cuda", dtype=BF), torch.zeros(H, tokens, device="cuda"), torch.zeros_like(qkv)]
    q, k, v = qkv.split(H * hd, 1)
    ws = xt.attention_masked_workspace(tokens, H, H, hd)
    torch.cuda.synchronize()

    def go():
        xt.xt_attention_masked_fwd(q, k, v, out[0], out[1], plan, H, H, hd, s=stream)
        xt.xt_attention_masked_bwd(q, k, v, out[0], do, out[1], *out[2].split(H * hd, 1), plan, H, H, hd, ws=ws, s=stream)
    return go, out


@pytest.mark.parametrize("hd", [64, 128])
def test_two_layers_of_one_plan_at_once(hd):
    """Many more work items than SMs, on two streams at the same time, sharing one plan: bit for bit the results of
    running alone."""
    tokens, H = 3000, 16
    plan = xt.attention_plan_buffer(tokens)
    xt.xt_attention_plan(plan, tokens, 5)
    alone = []
    for seed in (1, 2):
        go, out = attention_run(seed, plan, tokens, H, hd)
        go()
        torch.cuda.synchronize()
        alone.append(out)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    runs = [attention_run(seed, plan, tokens, H, hd, st) for seed, st in zip((1, 2), s)]
    for _ in range(3):
        for go, _out in runs:
            go()
    torch.cuda.synchronize()
    assert xt.device_errors() == 0
    for (_go, out), want in zip(runs, alone):
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("hd", [64, 128])
def test_waits_run_out_then_recover(hd):
    """With a limit of 1 ns the first wait that is not already satisfied runs out: the flag is set, the call returns,
    and after the flag is cleared and the limit restored the same call gives the same results bit for bit."""
    tokens, H = 700, 2
    plan = xt.attention_plan_buffer(tokens)
    xt.xt_attention_plan(plan, tokens, 1)
    go, out = attention_run(3, plan, tokens, H, hd)
    go()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    assert xt.device_errors() == 0
    try:
        xt.set_wait_limit_ns(1)
        go()
        torch.cuda.synchronize()
        assert xt.device_errors() & xt.XT_DEVERR_TIMEOUT
    finally:
        xt.set_wait_limit_ns(0)
        xt.clear_device_errors()
    go()
    torch.cuda.synchronize()
    assert xt.device_errors() == 0
    assert all(torch.equal(a, b) for a, b in zip(out, want))
