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


@pytest.mark.parametrize("hd,Hkv", [(64, 2), (128, 2), (64, 1)])
@pytest.mark.parametrize("y", [7.0, 8.0, -8.0, 10.0])
def test_gradients_of_saturated_scores(y, hd, Hkv):
    """Every score near y times the cap, where 1 − tanh² is 4e-6 to 8e-9 and the difference 1 − t·t of float32 numbers
    is off by 2⁻²⁴.  As in Case.reference, but every error of dS is relative to the factor too:
      dS    2⁻⁸ |dS| for its own rounding, 2⁻¹¹ |dS| for the factor's storage in 11 bits, 2(δ + 2⁻²⁰) |dS| for the error δ
            of y in it (d ln(1 − t²)/dy = −2t) and its exponential,
      W     the same factor beside D's correction;
      dP    hd·2⁻²⁴ Σ|dO v| in float32, and what that adds up to in D."""
    H, cap = 2, 1.0
    off = [0, 3, 10, 40, 41, 140]
    c = Case(off=off, H=H, Hkv=Hkv, hd=hd, cap=cap)
    q, k, _ = c.split(c.qkv)
    g = torch.Generator(device="cuda").manual_seed(11)
    near = lambda t, at: t.copy_(at + 0.05 * torch.randn(t.shape, generator=g, device="cuda"))  # noqa: E731
    a = math.sqrt(abs(y) / math.sqrt(hd))
    near(q, math.copysign(a, y))
    near(k, a)
    got = c.run()
    q, k, v = (t.double().view(c.T, -1, hd) for t in c.split(c.qkv))
    do, scale = c.do.double().view(c.T, H, hd), 1.0 / math.sqrt(hd)
    val = {n: torch.zeros(c.T, m, hd, dtype=torch.float64, device="cuda") for n, m in (("dq", H), ("dk", Hkv))}
    tol = {n: torch.zeros_like(t) for n, t in val.items()}
    for b, e in zip(off, off[1:]):
        at, see = slice(b, e), c.visible(e - b, 0)
        for h in range(H):
            kh = h // (H // Hkv)
            Q, K, V, G = q[at, h], k[at, kh], v[at, kh], do[at, h]
            x = Q @ K.T * scale / cap
            delta = hd * 2.0 ** -24 * (Q.abs() @ K.abs().T) * scale / cap + 2.0 ** -22 * x.abs()
            s = (cap * torch.tanh(x)).masked_fill(~see, -math.inf)
            P = torch.softmax(s, 1)
            slack = 1.0 / torch.cosh(x).square()
            dP = G @ V.T
            D = (P * dP).sum(1, keepdim=True)
            dS = P * (dP - D) * slack
            dPe = hd * 2.0 ** -24 * (G.abs() @ V.abs().T)
            dPe = dPe + (P * dPe).sum(1, keepdim=True)
            E = 2.0 ** -19 + 2 * (2.0 ** -21 * cap)   # float32 terms and the scores' resolution, as E of Case.reference
            dSe = dS.abs() * (B8 + 2.0 ** -11 + 2 * (delta + 2.0 ** -20)) + P * slack * (E * (dP.abs() + D.abs()) + dPe)
            o = P @ V
            oerr = ((B8 + E) * P) @ V.abs() + B8 * o.abs()
            dQe = dSe + 2 * B8 * P * slack * (G.abs() * oerr).sum(1, keepdim=True)
            val["dq"][at, h] = scale * dS @ K
            tol["dq"][at, h] = scale * dQe @ K.abs()
            val["dk"][at, kh] += scale * dS.T @ Q
            tol["dk"][at, kh] += scale * dSe.T @ Q.abs()
    for n in val:
        v64 = val[n].reshape(c.T, -1)
        over = (got[n].double() - v64).abs() / (tol[n].reshape(c.T, -1) + B8 * v64.abs()).clamp_min(1e-30)
        assert float(over.max()) <= 1.0, (n, float(over.max()))


@pytest.mark.parametrize("hd", [64, 128])
def test_short_documents_carry_what_the_rounding_of_ds_left(hd):
    """Texts inside a tile have edge tiles alone, whose dS is multiplied with its remainder, so that dQ and dK are off by
    their own rounding only.  Of a normal variable that is 1.66e-3 of the norm (half a step is 2⁻⁸ at most; the mean
    square over a binade's mantissas); one bf16 of dS adds as much again, independent of it: 2.35e-3."""
    off = [0]
    while off[-1] < 2000:
        off.append(off[-1] + 5 + 7 * len(off) % 31)
    c = Case(off=off, H=4, hd=hd, seed=3)
    got = c.run()
    val, _ = c.reference()
    for n in ("dq", "dk"):
        e = float((got[n].double() - val[n]).norm() / val[n].norm())
        assert e <= 2.0e-3, (n, e)


def busy(stream):
    """Some 20 ms of work on `stream`: what is queued behind it has not begun when the host goes on."""
    with torch.cuda.stream(stream):
        x = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
        for _ in range(30):
            x = x @ x * 0.0
    return x


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_workspaces_of_calls_on_another_stream(raw):
    """ws = None and s = a busy stream: tensors that the current stream allocates after the call are its own."""
    side = torch.cuda.Stream()
    s = side.cuda_stream if raw else side
    T, H, hd = 2000, 2, 64
    c = Case(off=[0, 700, T], H=H, hd=hd)
    want, plan = c.run(), c.plan()
    q, k, v = c.split(c.qkv)
    d = torch.zeros_like(c.qkv)
    g = torch.randn(4_000_000, device="cuda")
    P = [[torch.ones_like(g)] for _ in range(2)]
    st = [xt.adamw8_state(p) for p in P]
    cfg = xt.adamw_config(1e-2, max_grad_norm=1.0, step=1)
    xt.xt_adamw8_step(cfg, P[0], [g], *st[0])
    nbytes = (xt.attention_masked_workspace(T, H, H, hd).numel(), xt.adamw8_workspace([g.numel()]).numel())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = busy(side)
    xt.xt_attention_masked_bwd(q, k, v, want["o"], c.do, want["lse"], *c.split(d), plan, H, H, hd, s=s)
    xt.xt_adamw8_step(cfg, P[1], [g], *st[1], s=s)
    mine = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in nbytes * 4]
    torch.cuda.synchronize()
    assert xt.device_errors() == 0 and bool(torch.isfinite(held).all())
    assert all(bool((t == 0x5A).all()) for t in mine)
    assert all(torch.equal(a, want[n]) for a, n in zip(c.split(d), ("dq", "dk", "dv")))
    assert torch.equal(P[0][0], P[1][0])


@pytest.mark.parametrize("shadow", [False, True], ids=["", "bf16-copy"])
@pytest.mark.parametrize("eps", [1e-16, 1e-20, 1e-30, 1e-42])
def test_adamw8_with_a_tiny_epsilon(eps, shadow):
    """Second moments whose root matters beside ε: roots down to 1e-19 and an ε below float32's normal range.  First step, so
    m' = (1 − β₁) g, v' = ((1 − β₂) g)·g; the update lr·m̂/(√v̂ + ε) carries 16·2⁻²⁴ of itself (m' 2 roundings, √v' 4, two
    bias factors, root, quotient and sum), v' of at least 2⁻¹²⁶ being a normal number."""
    g0 = np.concatenate([np.exp(np.linspace(math.log(6e-19), math.log(1e-15), 700)), np.zeros(100), [3e-5] * 224])
    g0 = (g0 * np.where(np.arange(g0.size) % 3 == 1, -1, 1)).astype(np.float32)
    p0 = np.where(np.arange(g0.size) < 700, 0.0, 0.5).astype(np.float32)
    P, G = [torch.from_numpy(p0).cuda()], [torch.from_numpy(g0).cuda()]
    S = [torch.zeros(p0.size, dtype=torch.bfloat16, device="cuda")] if shadow else None
    b1, b2 = float(np.float32(0.9)), float(np.float32(0.95))
    xt.xt_adamw8_step(xt.adamw_config(1e-3, beta1=0.9, beta2=0.95, eps=eps, weight_decay=0.1, step=1), P, G,
                      *xt.adamw8_state(P), shadows=S)
    g = g0.astype(np.float64)
    m, v, e = (1 - b1) * g, (1 - b2) * g * g, float(np.float32(eps))
    step = 1e-3 * (m / (1 - b1)) / (np.sqrt(v / (1 - b2)) + e)
    got, want = P[0].double().cpu().numpy(), p0 * (1 - 1e-4) - step
    # θ's own roundings: 3·2⁻²⁴ of its value (1 − lr·λ, the product, the sum)
    assert np.all(np.abs(got - want) <= 16 * 2.0 ** -24 * np.abs(step) + 3 * 2.0 ** -24 * np.abs(want))
    assert S is None or torch.equal(S[0], P[0].to(torch.bfloat16))


def test_train_step_losses_on_a_busy_stream():
    """The losses that train_step returns are copied on its stream, behind the forward that writes them."""
    import synth
    from transformer_fwd_bwd_gb300.block import NativeBlock
    cfg = dict(synth.BLOCK_CONFIGS["gpt12"], B=1, S=64, d=64, H=1, hd=64, F=128, V=256, n_layers=1)
    ids, tgt = (torch.from_numpy(a).cuda() for a in synth.block_tokens(cfg))
    side, out = torch.cuda.Stream(), []
    for s in (None, side):
        nb = NativeBlock(cfg, device="cuda:0", training=True)
        nb.load(synth.block_params(cfg))
        nb.init_optimizer(lr=1e-2, state_bits=8)
        torch.cuda.synchronize()
        held = busy(side)
        losses = nb.train_step([(ids, tgt), (ids.flip(0), tgt)], stream=s)
        torch.cuda.synchronize()
        out.append([float(x) for x in losses])
    assert out[0] == out[1] and bool(torch.isfinite(held).all())


def test_tape_rope_axes_refuses_columns_beside_the_heads():
    """xt_rope_axes_fwd rotates the first H·hd columns; a node's value and gradient are whole tensors."""
    from transformer_fwd_bwd_gb300 import tape
    pos = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    x = torch.ones(8, 3 * 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        tape.rope_axes(tape.leaf(x), pos, [8, 24], 2, 64)
    y = tape.rope_axes(tape.leaf(x), pos, [8, 24], 3, 64)
    assert torch.equal(y.value, x)   # position 0
