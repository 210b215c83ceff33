"""GPU parity of masked attention (xt_attention_plan, xt_attention_masked_fwd / _bwd) against its definition
in float64, document by document.

Tolerances, element by element, from the roundings the kernels make (bf16: half a step, 2⁻⁸ relative):
  O    P is rounded before it multiplies V, O when it is stored:     2⁻⁸ (Σ_j P|v_j| + |O|)
  dV   the same of Pᵀ and dV:                                       2⁻⁸ (Σ_i P|dO_i| + |dV|)
  dS   is rounded itself:                                           2⁻⁸ |dS|; dQ and dK sum it against |k| and
       |q| and round once.  D is summed in float32 from P and dP (the stored O's rounding cancels): dQ is the sum of
       dS₀ = P(1 − t²)(dP − D₀) less T = D − D₀ times the sum of W = P(1 − t²), both rounded to bf16: 2⁻⁸ |dS₀| and
       2⁻⁸ W|T|, with |T| ≤ 2⁻⁸ Σ_c |dO_c| (Σ_j P|v_jc| + |O_c|) (P's and O's rounding in D₀ = dO·O).
float32 arithmetic adds, relative to the terms P|v|, P|dO| and P(|dP| + |D|): the scores' own error, at most
hd·2⁻²⁴ Σ|q k| scale (and 2⁻²¹ cap), and 2⁻²⁰ for exponential, quotient and sums — `E` below."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_util import empty

pytestmark = pytest.mark.gpu

xt = pytest.importorskip("transformer_fwd_bwd_gb300.xt")

B8 = 2.0 ** -8


class Case:
    def __init__(self, off, hd=64, H=2, Hkv=None, causal=1, lens=None, prefix=None, cap=0.0, bias=False, scale=None,
                 qstd=1.5, seed=1, T=None):
        self.off, self.hd, self.H, self.Hkv, self.causal = list(off), hd, H, Hkv or H, causal
        self.T = T if T is not None else self.off[-1]
        n = len(self.off) - 1
        self.lens = list(lens) if lens is not None else [self.off[i + 1] - self.off[i] for i in range(n)]
        self.has_len = lens is not None
        self.prefix = list(prefix) if prefix is not None else None
        self.cap, self.scale = cap, scale
        g = torch.Generator(device="cuda").manual_seed(seed)
        W = (H + 2 * self.Hkv) * hd
        qkv = torch.randn(self.T, W, generator=g, device="cuda")
        qkv[:, :H * hd] *= qstd
        self.qkv = qkv.to(torch.bfloat16)
        self.do = torch.randn(self.T, H * hd, generator=g, device="cuda").to(torch.bfloat16)
        self.slopes = torch.exp2(-torch.arange(1, H + 1, device="cuda").float()) if bias else None

    def split(self, t):
        return t.split([self.H * self.hd, self.Hkv * self.hd, self.Hkv * self.hd], dim=1)

    def plan(self):
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda") if v is not None else None  # noqa: E731
        plan = xt.attention_plan_buffer(self.T)
        self.arrays = ints(self.off), ints(self.lens) if self.has_len else None, ints(self.prefix)
        xt.xt_attention_plan(plan, self.T, len(self.off) - 1, *self.arrays, causal=self.causal)
        return plan

    def run(self, backward=True):
        T, H, Hkv, hd = self.T, self.H, self.Hkv, self.hd
        plan = self.plan()
        q, k, v = self.split(self.qkv)
        o, lse = empty((T, H * hd), "bf16", fill=7.0), empty((H, T), fill=7.0)
        kw = dict(scale=self.scale, cap=self.cap, slopes=self.slopes)
        xt.xt_attention_masked_fwd(q, k, v, o, lse, plan, H, Hkv, hd, **kw)
        out = {"o": o, "lse": lse}
        if backward:
            d = empty((T, (H + 2 * Hkv) * hd), "bf16", fill=7.0)
            dq, dk, dv = self.split(d)
            xt.xt_attention_masked_bwd(q, k, v, o, self.do, lse, dq, dk, dv, plan, H, Hkv, hd, **kw)
            out |= {"dq": dq, "dk": dk, "dv": dv}
        torch.cuda.synchronize()
        assert xt.device_errors() == 0
        return out

    def visible(self, m, pl):
        i = torch.arange(m, device="cuda")
        if not self.causal:
            return torch.ones(m, m, dtype=torch.bool, device="cuda")
        return (i[None, :] <= i[:, None]) | (i < pl)[None, :]

    def reference(self, forward_only=False, qkv=None):
        """Values and tolerances in float64."""
        T, H, Hkv, hd = self.T, self.H, self.Hkv, self.hd
        scale = self.scale or 1.0 / math.sqrt(hd)
        z = lambda n: torch.zeros(T, n, hd, dtype=torch.float64, device="cuda")  # noqa: E731
        q, k, v = (t.double().view(T, -1, hd) for t in self.split(self.qkv if qkv is None else qkv))
        do = self.do.double().view(T, H, hd)
        val = {"o": z(H), "dq": z(H), "dk": z(Hkv), "dv": z(Hkv),
               "lse": torch.full((H, T), -math.inf, dtype=torch.float64, device="cuda")}
        tol = {n: torch.zeros_like(t) for n, t in val.items()}
        for d in range(len(self.off) - 1):
            a, m = self.off[d], self.lens[d]
            if m == 0:
                continue
            at = slice(a, a + m)
            see = self.visible(m, min(self.prefix[d], m) if self.prefix else 0)
            i = torch.arange(m, device="cuda")
            for h in range(H):
                kh = h // (H // Hkv)
                Q, K, V, G = q[at, h], k[at, kh], v[at, kh], do[at, h]
                s = Q @ K.T * scale
                se = hd * 2.0 ** -24 * (Q.abs() @ K.abs().T) * scale   # error of a float32 score
                slack = torch.ones_like(s)
                if self.cap:
                    t = torch.tanh(s / self.cap)
                    s, slack = self.cap * t, 1 - t * t
                    se = se + 2.0 ** -21 * self.cap
                if self.slopes is not None:
                    b = float(self.slopes[h]) * (i[:, None] - i[None, :]).abs()
                    s = s - b
                    se = se + 2.0 ** -22 * b   # slope·log₂e and the product round
                s = s.masked_fill(~see, -math.inf)
                lse = torch.logsumexp(s, 1)
                P = torch.exp(s - lse[:, None])
                se = se.masked_fill(~see, 0.0)
                E = se + se.amax(1, keepdim=True) + 2.0 ** -20 + 2.0 ** -23 * (s.masked_fill(~see, 0.0).abs() + lse.abs()[:, None])
                val["lse"][h, at] = lse
                tol["lse"][h, at] = E.amax(1) + 2.0 ** -22 * lse.abs()
                val["o"][at, h] = P @ V
                te = (B8 + E) * P
                oerr = te @ V.abs()
                tol["o"][at, h] = oerr + B8 * val["o"][at, h].abs()
                if forward_only:
                    continue
                val["dv"][at, kh] += P.T @ G
                tol["dv"][at, kh] += te.T @ G.abs()
                dP = G @ V.T
                D = (P * dP).sum(1, keepdim=True)
                dS = P * (dP - D) * slack
                tmax = (G.abs() * (oerr + B8 * val["o"][at, h].abs())).sum(1, keepdim=True)
                dSe = B8 * dS.abs() + E * P * (dP.abs() + D.abs()) + P * se * 2 * (dP.abs() + D.abs()) / max(self.cap, 1.0)
                dQe = dSe + 2 * B8 * P * slack * tmax
                val["dq"][at, h] = scale * dS @ K
                tol["dq"][at, h] = scale * dQe @ K.abs()
                val["dk"][at, kh] += scale * dS.T @ Q
                tol["dk"][at, kh] += scale * dSe.T @ Q.abs()
        for n in ("dq", "dk", "dv"):
            tol[n] = tol[n] + B8 * val[n].abs()
        flat = lambda t: t if t.shape[0] == H and t.dim() == 2 else t.reshape(T, -1)  # noqa: E731
        return {n: flat(t) for n, t in val.items()}, {n: flat(t) for n, t in tol.items()}


def compare(got, val, tol, names=("o", "lse", "dq", "dk", "dv")):
    for n in names:
        g, w = got[n].double(), val[n]
        fin = torch.isfinite(w)
        assert torch.equal(torch.isfinite(g), fin), n
        assert torch.equal(g[~fin], w[~fin]), n
        # accumulated and stored in float32 before the one rounding: 1e-30 lets exact zeros be zeros
        over = ((g - w).abs() - tol[n])[fin]
        if over.numel():
            k = int(over.argmax())
            assert float(over.max()) <= 1e-30, (n, float(over.max()), float(w[fin][k]), float(tol[n][fin][k]))


CASES = {
    "one-token": dict(off=[0, 1], H=1),
    "one-text": dict(off=[0, 77], H=3),
    "one-text-128": dict(off=[0, 128], H=1, hd=128),
    "tile-plus-one": dict(off=[0, 129], H=2, hd=128),
    "three-tiles": dict(off=[0, 384], H=2),
    "packed": dict(off=[0, 100, 100, 101, 229, 400, 611], H=2),
    "packed-128": dict(off=[0, 100, 100, 101, 229, 400, 611], H=2, hd=128),
    "tiny-documents": dict(off=list(range(0, 200, 3)) + [200], H=1),
    "shared-heads": dict(off=[0, 150, 300], H=6, Hkv=2),
    "shared-heads-128": dict(off=[0, 150, 420], H=8, Hkv=1, hd=128),
    "images": dict(off=[0, 196, 300, 556], H=2, causal=0),
    "images-128": dict(off=[0, 196, 300, 556], H=4, Hkv=2, hd=128, causal=0),
    "prefix": dict(off=[0, 300, 500], H=2, prefix=[140, 999]),
    "prefix-128": dict(off=[0, 300, 500], H=2, hd=128, prefix=[129, 0]),
    "padded": dict(off=[0, 130, 260, 390], lens=[130, 1, 0], H=2),
    "padded-128": dict(off=[0, 200, 400], lens=[77, 199], H=2, hd=128, prefix=[50, 7]),
    "tail-outside": dict(off=[3, 200], H=2, T=333),
    "cap": dict(off=[0, 140, 270], H=2, cap=30.0, qstd=8.0),
    "cap-128": dict(off=[0, 140, 270], H=4, Hkv=2, hd=128, cap=50.0, qstd=8.0),
    "one-key-head": dict(off=[0, 200, 333], H=12, Hkv=1),
    "one-key-head-128": dict(off=[0, 77, 333], H=6, Hkv=1, hd=128, bias=True),
    "uneven-parts": dict(off=list(range(0, 9729, 128)), H=10, Hkv=2),  # five heads of a group in parts of 2, 2 and 1
    "cap-large": dict(off=[0, 140, 270], H=2, cap=1000.0, qstd=8.0),
    "cap-small": dict(off=[0, 200], H=1, cap=0.5, qstd=1.0),
    "bias": dict(off=[0, 140, 470], H=3, bias=True),
    "bias-128": dict(off=[0, 140, 470], H=3, hd=128, bias=True),
    "bias-images": dict(off=[0, 140, 470], H=2, bias=True, causal=0),
    "bias-prefix-cap": dict(off=[0, 333, 470], H=2, bias=True, prefix=[200, 10], cap=20.0, qstd=5.0),
    "bias-prefix-cap-128": dict(off=[0, 333, 470], H=4, Hkv=2, hd=128, bias=True, prefix=[200, 10], cap=20.0, qstd=5.0),
    "scale": dict(off=[0, 100, 200], H=2, scale=0.3),
    "large-scores": dict(off=[0, 512], H=2, qstd=20.0),
    "no-documents": dict(off=[0], H=1, T=140),
    "many-tiles": dict(off=[0, 700, 1500, 1501, 2900], H=2),
    "many-tiles-128": dict(off=[0, 1700, 2600], H=4, Hkv=2, hd=128),
}


@pytest.mark.parametrize("name", CASES)
def test_parity(name):
    c = Case(**CASES[name])
    val, tol = c.reference()
    compare(c.run(), val, tol)


def test_equal_spans_without_offsets():
    """doc_off = NULL: n_docs equal spans give what the offsets of the spans give."""
    c = Case(off=[0, 150, 300, 450], H=2)
    a = c.run()
    plan = xt.attention_plan_buffer(450)
    xt.xt_attention_plan(plan, 450, 3)
    q, k, v = c.split(c.qkv)
    o, lse = empty((450, 128), "bf16"), empty((2, 450))
    xt.xt_attention_masked_fwd(q, k, v, o, lse, plan, 2, 2, 64)
    assert torch.equal(o, a["o"]) and torch.equal(lse, a["lse"])


def test_reference_gradient_against_differences():
    """The formulas that the kernels are held to, against central differences of the reference's forward
    along a direction: truncation h²·f''' and rounding 2⁻⁵³/h leave 1e-7 at h = 1e-4."""
    c = Case(off=[0, 20, 33], H=2, Hkv=1, cap=3.0, bias=True, prefix=[7, 0], qstd=2.0)
    val, _ = c.reference()
    g = torch.Generator(device="cuda").manual_seed(5)
    u = torch.randn(*c.qkv.shape, generator=g, device="cuda", dtype=torch.float64)
    f = lambda h: float((c.reference(True, c.qkv.double() + h * u)[0]["o"] * c.do.double()).sum())  # noqa: E731
    num = (f(1e-4) - f(-1e-4)) / 2e-4
    d = torch.cat([val["dq"], val["dk"], val["dv"]], 1)
    assert abs(num - float((d * u).sum())) <= 1e-6 * float((d * u).abs().sum())


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_masked_values_that_are_not_finite(hd, bad):
    """NaN and infinities in padding and in one document: every other token's results are the definition's."""
    c = Case(off=[0, 90, 200, 330], lens=[80, 110, 130], H=2, Hkv=1, hd=hd, prefix=[0, 20, 40])
    val, tol = c.reference()
    for t in (c.qkv, c.do):
        t[80:90] = bad       # padding
        t[195] = bad         # near the end of document 1
    got = c.run()
    keep = torch.ones(330, dtype=torch.bool, device="cuda")
    keep[90:200] = False
    for n in ("o", "dq", "dk", "dv"):
        compare({n: got[n][keep]}, {n: val[n][keep]}, {n: tol[n][keep]}, (n,))
    compare({"lse": got["lse"][:, keep]}, {"lse": val["lse"][:, keep]}, {"lse": tol["lse"][:, keep]}, ("lse",))
    # document 1: rows before the bad token do not see its key or value
    early = slice(90, 195)
    compare({"o": got["o"][early]}, {"o": val["o"][early]}, {"o": tol["o"][early]}, ("o",))
    assert not bool(torch.isfinite(got["o"][195]).any())


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("first", [129, 130, 131, 132])
def test_capped_scores_beside_a_masked_nan(hd, first):
    """A document's first column beside the NaN of the last token before it, at each place among four columns."""
    c = Case(off=[0, first, 270], H=2, Hkv=1, hd=hd, cap=20.0)
    val, tol = c.reference()
    for t in (c.qkv, c.do):
        t[first - 1] = float("nan")
    got = c.run()
    keep = slice(first, 270)
    for n in ("o", "dq", "dk", "dv"):
        compare({n: got[n][keep]}, {n: val[n][keep]}, {n: tol[n][keep]}, (n,))
    early = slice(0, first - 1)  # causal: they do not see it, and no gradient of O comes from it
    compare({"o": got["o"][early]}, {"o": val["o"][early]}, {"o": tol["o"][early]}, ("o",))


def test_deterministic_strides_stream_and_capture():
    c = Case(off=[0, 300, 700], H=4, Hkv=2, hd=64, cap=20.0, bias=True)
    a = c.run()
    T, H, Hkv, hd = c.T, c.H, c.Hkv, c.hd
    plan = c.plan()
    # tensors of their own, with another row stride
    wide = lambda t, x: torch.cat([t, torch.full((T, x), 9.0, device="cuda", dtype=t.dtype)], 1)[:, :t.shape[1]]  # noqa: E731
    q, k, v = (wide(t, x) for t, x in zip(c.split(c.qkv), (8, 24, 40)))
    do = wide(c.do, 8)
    s = torch.cuda.Stream()
    outs = []
    for mode in ("stream", "graph"):
        o, lse = torch.zeros(T, H * hd + 16, device="cuda", dtype=torch.bfloat16), empty((H, T))
        dq, dk, dv = (torch.zeros(T, n * hd + x, device="cuda", dtype=torch.bfloat16) for n, x in ((H, 0), (Hkv, 8), (Hkv, 16)))
        ws = xt.attention_masked_workspace(T, H, Hkv, hd)
        views = o[:, :H * hd], dq, dk[:, :Hkv * hd], dv[:, :Hkv * hd]

        def both(st):
            kw = dict(cap=c.cap, slopes=c.slopes, s=st)
            xt.xt_attention_plan(plan, T, 2, *c.arrays, causal=1, s=st)
            xt.xt_attention_masked_fwd(q, k, v, views[0], lse, plan, H, Hkv, hd, **kw)
            xt.xt_attention_masked_bwd(q, k, v, views[0], do, lse, *views[1:], plan, H, Hkv, hd, ws=ws, **kw)
        torch.cuda.synchronize()
        if mode == "stream":
            both(s)
        else:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                both(None)
            g.replay()
            g.replay()
        torch.cuda.synchronize()
        for x, n in zip(views, ("o", "dq", "dk", "dv")):
            assert torch.equal(x, a[n]), (mode, n)
        assert torch.equal(lse, a["lse"])
        assert not bool(o[:, H * hd:].any()) and not bool(dk[:, Hkv * hd:].any()) and not bool(dv[:, Hkv * hd:].any())
        outs.append((o, dq, dk, dv))
    assert xt.device_errors() == 0


def test_plan_of_another_batch_is_refused_on_the_device():
    c = Case(off=[0, 300], H=1)
    q, k, v = c.split(c.qkv)
    plan = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    xt.xt_attention_plan(plan, 260, 1)
    o, lse = empty((300, 64), "bf16", fill=3.0), empty((1, 300), fill=3.0)
    xt.xt_attention_masked_fwd(q, k, v, o, lse, plan, 1, 1, 64)
    try:
        assert xt.device_errors() == xt.XT_DEVERR_PLAN
        assert bool((o == 3.0).all()) and bool((lse == 3.0).all())
    finally:
        xt.clear_device_errors()


def test_bad_documents_are_reported():
    T = 300
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for args in ((ints([0, 200, 100]), None, None), (ints([0, 100, 400]), None, None), (ints([-5, 100, 300]), None, None),
                 (ints([0, 100, 300]), ints([101, 5]), None), (ints([0, 100, 300]), ints([-1, 5]), None),
                 (ints([0, 100, 300]), None, ints([0, -2]))):
        plan = xt.attention_plan_buffer(T)
        xt.xt_attention_plan(plan, T, 2, *args)
        try:
            assert xt.device_errors() == xt.XT_DEVERR_INDEX
        finally:
            xt.clear_device_errors()


def test_long_text():
    """More key tiles than any ring holds; the work order of 64 tiles; shared heads."""
    c = Case(off=[0, 5000, 8100], H=2, Hkv=1, hd=128, cap=30.0, qstd=4.0)
    val, tol = c.reference()
    compare(c.run(), val, tol)


def test_offsets_beyond_32_bits():
    """The last of 1024 texts, whose elements lie behind 2^32, gives what it gives alone, bit for bit."""
    T, n, H, hd = 1 << 20, 1024, 16, 128
    d = H * hd
    g = torch.Generator(device="cuda").manual_seed(5)
    last = torch.randn(n, 4 * d, generator=g, device="cuda").to(torch.bfloat16)

    def run(T):
        qkvg = torch.zeros(T, 4 * d, dtype=torch.bfloat16, device="cuda")
        qkvg[-n:] = last
        q, k, v, do = qkvg.split(d, 1)
        out = torch.full((T, 4 * d), 7.0, dtype=torch.bfloat16, device="cuda")
        o, dq, dk, dv = out.split(d, 1)
        lse = torch.full((H, T), 7.0, device="cuda")
        plan = xt.attention_plan_buffer(T)
        xt.xt_attention_plan(plan, T, T // n)
        xt.xt_attention_masked_fwd(q, k, v, o, lse, plan, H, H, hd)
        xt.xt_attention_masked_bwd(q, k, v, o, do, lse, dq, dk, dv, plan, H, H, hd)
        torch.cuda.synchronize()
        assert xt.device_errors() == 0
        return out[-n:].clone(), lse[:, -n:].clone(), out[:n].clone()

    alone, far = run(n), run(T)
    assert torch.equal(alone[0], far[0]) and torch.equal(alone[1], far[1])
    assert not bool(far[2].any())   # the first text is all zeros


@pytest.mark.parametrize("hd,H,Hkv", [(64, 2, 2), (128, 2, 2), (64, 4, 1)])
@pytest.mark.parametrize("T", [1, 31, 97, 200])
def test_outputs_touch_nothing_else(T, hd, H, Hkv):
    """Outputs inside a larger buffer: the columns beside and the rows behind them stay as they were."""
    W, pad, rows = (2 * H + 2 * Hkv) * hd, 64, T + 70
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k, v, do = torch.randn(T, W, generator=g, device="cuda").to(torch.bfloat16).split([H * hd, Hkv * hd, Hkv * hd, H * hd], 1)
    buf = torch.full((rows, W + 2 * pad), 7.0, dtype=torch.bfloat16, device="cuda")
    o, dq, dk, dv = buf[:T, pad:pad + W].split([H * hd, H * hd, Hkv * hd, Hkv * hd], 1)
    lse = torch.empty(H, T, device="cuda")
    plan = xt.attention_plan_buffer(T)
    xt.xt_attention_plan(plan, T, 1)
    xt.xt_attention_masked_fwd(q, k, v, o, lse, plan, H, Hkv, hd)
    for outs, done in (((o,), [o]), ((dq, dk, dv), [o, dq, dk, dv])):
        if len(outs) > 1:
            xt.xt_attention_masked_bwd(q, k, v, o, do, lse, dq, dk, dv, plan, H, Hkv, hd)
        mark = torch.zeros_like(buf, dtype=torch.bool)
        for t in done:
            c = (t.data_ptr() - buf.data_ptr()) // 2
            mark[:T, c:c + t.shape[1]] = True
        assert bool((buf[~mark] == 7.0).all())
    assert xt.device_errors() == 0
