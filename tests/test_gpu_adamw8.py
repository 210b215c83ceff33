"""GPU parity of the AdamW step with 8-bit moments (xt_adamw8_step, xt_adamw8_decode) against its
definition, evaluated in float32 with every operation rounded by itself (NumPy's float32 arithmetic): codes
and scales are equal bit for bit.  The weights are held to the float64 update of the unrounded moments:
lr·|m̂|/(√v̂ + ε) is formed with relative error below 16·2⁻²⁴ (m' 3 roundings, √v' 4, two bias factors, an
approximate root, quotient and sum), θ(1 − lrλ) and the difference round once each; where (1−β₁)g' and β₁m
cancel, the error of m' is relative to the larger."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

xt = pytest.importorskip("transformer_fwd_bwd_gb300.xt")

HP = dict(lr=2e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
F = np.float32
BLOCK = 256


def blocks(x):
    n = -(-x.size // BLOCK)
    out = np.zeros(n * BLOCK, x.dtype)
    out[:x.size] = x
    return out.reshape(n, BLOCK)


class Reference:
    def __init__(self, p):
        self.p = p.astype(np.float64)
        n = -(-p.size // BLOCK)
        self.cm, self.cr = np.zeros(p.size, np.int32), np.zeros(p.size, np.int32)
        self.ms, self.rs = np.zeros(n, F), np.zeros(n, F)
        self.tol = np.zeros(p.size)

    def moments(self):
        per = np.repeat(self.ms, BLOCK)[:self.cm.size], np.repeat(self.rs, BLOCK)[:self.cm.size]
        m = (self.cm * np.abs(self.cm)).astype(F) * per[0]
        r = (self.cr * self.cr).astype(F) * per[1]
        return m, r * r

    def step(self, g, f, t):
        b1, b2 = F(HP["beta1"]), F(HP["beta2"])
        o1, o2 = F(1) - b1, F(1) - b2
        m0, v0 = self.moments()
        with np.errstate(all="ignore"):
            gg = g * F(f)
            m = m0 * b1 + gg * o1
            v = v0 * b2 + (gg * o2) * gg
            g64 = g.astype(np.float64) * float(F(f))
            m64 = float(b1) * m0 + float(o1) * g64
            v64 = float(b2) * v0.astype(np.float64) + float(o2) * g64 * g64
            lr, wd, eps = HP["lr"], HP["weight_decay"], HP["eps"]
            bc1, bc2 = 1 - float(b1) ** t, 1 - float(b2) ** t
            den = np.sqrt(v64 / bc2) + eps
            self.p = self.p * (1 - lr * wd) - lr * (m64 / bc1) / den
            big = lr * ((np.abs(float(b1) * m0) + np.abs(float(o1) * g64)) / bc1) / den
            self.tol = self.tol + 16 * 2.0 ** -24 * big + 3 * 2.0 ** -24 * (np.abs(self.p) + big)
            am, r = blocks(np.abs(m)), blocks(np.sqrt(v))
            self.ms, self.rs = am.max(1) / F(16129), r.max(1) / F(65025)
            code = lambda x, s: np.where((s > 0) & np.isfinite(s), np.rint(np.sqrt(x / s)), F(0))  # noqa: E731
            cm, cr = code(am, self.ms[:, None]), code(r, self.rs[:, None])
            cm, cr = cm.reshape(-1)[:g.size], cr.reshape(-1)[:g.size]
            ok = np.isfinite(np.repeat(self.rs, BLOCK)[:g.size]) & (np.repeat(self.rs, BLOCK)[:g.size] > 0)
            cr = np.where((v > 0) & ok, np.maximum(cr, F(1)), cr)
        self.cm = np.where(m < 0, -cm, cm).astype(np.int32)
        self.cr = cr.astype(np.int32)


def upload(a, offset):
    """The array on the GPU, `offset` elements behind an aligned start."""
    t = torch.from_numpy(np.ascontiguousarray(a))
    buf = torch.zeros(t.numel() + offset, dtype=t.dtype, device="cuda")
    buf[offset:] = t.cuda()
    return buf[offset:]


def factor(grads, scale, max_norm):
    norm = abs(scale) * math.sqrt(math.fsum(float(np.sum(g.astype(np.float64) ** 2)) for g in grads))
    c = min(1.0, max_norm / (norm + 1e-6)) if max_norm > 0 else 1.0
    return float(F(scale * c)), norm


def run(sizes, steps, max_norm=0.0, scale=1.0, offset=0, gscale=1.0, shadow=None, seed=0):
    rng = np.random.default_rng(seed)
    p = [rng.normal(size=n).astype(F) * F(0.05) for n in sizes]
    ref = [Reference(x) for x in p]
    P = [upload(x, offset) for x in p]
    M, R, MS, RS = xt.adamw8_state(P)
    if offset:
        M, R = [upload(t.cpu().numpy(), offset) for t in M], [upload(t.cpu().numpy(), offset) for t in R]
    S = [torch.zeros(n, dtype=shadow, device="cuda") for n in sizes] if shadow else None
    norm = torch.zeros(1, device="cuda")
    for t in range(1, steps + 1):
        g = [(rng.normal(size=n) * np.exp(rng.normal(size=n) * 2) * gscale).astype(F) for n in sizes]
        f, want = factor(g, scale, max_norm)
        cfg = xt.adamw_config(step=t, max_grad_norm=max_norm, grad_scale=scale, **HP)
        xt.xt_adamw8_step(cfg, P, [upload(x, offset) for x in g], M, R, MS, RS, shadows=S, norm_out=norm)
        assert abs(float(norm.item()) - want) <= 2.0 ** -23 * want
        for r, x in zip(ref, g):
            r.step(x, f, t)
        for i, r in enumerate(ref):
            assert np.array_equal(MS[i].cpu().numpy(), r.ms) and np.array_equal(RS[i].cpu().numpy(), r.rs), (t, i)
            assert np.array_equal(M[i].cpu().numpy().astype(np.int32), r.cm), (t, i)
            assert np.array_equal(R[i].cpu().numpy().astype(np.int32), r.cr), (t, i)
            assert np.all(np.abs(P[i].cpu().numpy() - r.p) <= r.tol), (t, i)
            if S:
                assert torch.equal(S[i], P[i].to(shadow))
    m, v = [torch.empty(n, device="cuda") for n in sizes], [torch.empty(n, device="cuda") for n in sizes]
    xt.xt_adamw8_decode(M, R, MS, RS, m, v)
    for i, r in enumerate(ref):
        a, b = r.moments()
        assert np.array_equal(m[i].cpu().numpy(), a) and np.array_equal(v[i].cpu().numpy(), b)
    assert xt.device_errors() == 0


SIZES = [1, 255, 256, 0, 257, 4096, 4097, 10007, 777]


@pytest.mark.parametrize("max_norm,scale", [(0.0, 1.0), (1.0, 0.5), (1e9, 0.25)],
                         ids=["no-clip", "clip-active", "clip-inactive"])
def test_parity(max_norm, scale):
    run(SIZES, 4, max_norm, scale)


def test_bf16_working_copy_and_many_tensors():
    """More tensors than one launch takes, the norm over all of them."""
    run([1 + 37 * i % 900 for i in range(300)], 2, 1.0, 0.5, shadow=torch.bfloat16)


@pytest.mark.parametrize("offset", [1, 4])
def test_misaligned_tensors(offset):
    run([5000, 513], 2, 1.0, 1.0, offset=offset, shadow=torch.float32)


@pytest.mark.parametrize("gscale", [1e-22, 1e-18, 1e-12, 1e15])
def test_far_magnitudes(gscale):
    """Gradients whose squares leave float32's normal range, or nearly do."""
    run([600, 4096], 2, 0.0, 1.0, gscale=gscale)


def test_large_tensor_codes():
    """Enough elements that some lie next to a border between codes."""
    run([3000001], 2, 1.0, 1.0, seed=3)


def test_zero_gradients_keep_zero_state():
    P = [torch.ones(1000, device="cuda")]
    st = xt.adamw8_state(P)
    cfg = xt.adamw_config(step=1, max_grad_norm=1.0, **HP)
    norm = torch.ones(1, device="cuda")
    xt.xt_adamw8_step(cfg, P, [torch.zeros(1000, device="cuda")], *st, norm_out=norm)
    assert float(norm) == 0.0 and all(not bool(t[0].any()) for t in st)
    assert torch.equal(P[0], torch.ones(1000, device="cuda") * F(1 - HP["lr"] * HP["weight_decay"]))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_gradient_that_is_not_finite_stays_in_its_block(bad):
    P = [torch.ones(1024, device="cuda")]
    st = xt.adamw8_state(P)
    g = torch.full((1024,), 0.01, device="cuda")
    g[300] = bad
    xt.xt_adamw8_step(xt.adamw_config(step=1, **HP), P, [g], *st)
    m, v = [torch.empty(1024, device="cuda")], [torch.empty(1024, device="cuda")]
    xt.xt_adamw8_decode(*st, m, v)
    for t in (m[0], v[0]):
        assert bool(torch.isfinite(t[:256]).all()) and bool(torch.isfinite(t[512:]).all())
        assert not bool(torch.isfinite(t[300]))
    assert bool(torch.isfinite(P[0][:300]).all()) and not bool(torch.isfinite(P[0][300]))


def test_capture_and_other_stream():
    rng = np.random.default_rng(9)
    g = torch.tensor(rng.normal(size=5000).astype(F), device="cuda")
    outs = []
    for mode in ("plain", "stream", "graph"):
        P = [torch.ones(5000, device="cuda")]
        st = xt.adamw8_state(P)
        ws = xt.adamw8_workspace([5000])
        cfg = xt.adamw_config(step=1, max_grad_norm=1.0, **HP)
        torch.cuda.synchronize()
        if mode == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                xt.xt_adamw8_step(cfg, P, [g], *st, ws=ws)
            graph.replay()
        elif mode == "stream":
            s = torch.cuda.Stream()
            xt.xt_adamw8_step(cfg, P, [g], *st, ws=ws, s=s)
        else:
            xt.xt_adamw8_step(cfg, P, [g], *st, ws=ws)
        torch.cuda.synchronize()
        outs.append([P[0], st[0][0], st[1][0], st[2][0], st[3][0]])
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_norm_of_empty_tensors():
    """No tile at all, and no workspace: the norm is still reported."""
    P = [torch.empty(0, device="cuda") for _ in range(2)]
    st = xt.adamw8_state(P)
    norm = torch.full((1,), 7.0, device="cuda")
    xt.xt_adamw8_step(xt.adamw_config(step=1, max_grad_norm=1.0, **HP), P, [torch.empty_like(p) for p in P], *st,
                      norm_out=norm)
    assert float(norm) == 0.0


def test_host_tensors_are_refused():
    P = [torch.ones(300, device="cuda")]
    st, cfg = xt.adamw8_state(P), xt.adamw_config(step=1, **HP)
    host = [torch.zeros(300)]
    for kw in (dict(shadows=host), dict(shadows=[torch.zeros(299, device="cuda")]),
               dict(shadows=[torch.zeros(300, device="cuda", dtype=torch.float16)])):
        with pytest.raises((ValueError, TypeError)):
            xt.xt_adamw8_step(cfg, P, [torch.zeros_like(P[0])], *st, **kw)
    with pytest.raises(ValueError):
        xt.xt_adamw8_step(cfg, P, host, *st)
    with pytest.raises(ValueError):
        xt.xt_adamw8_decode(*st, m=host)
    with pytest.raises(ValueError):
        xt.xt_adamw8_decode(*st, v=[torch.zeros(300, device="cuda"), P[0]])
