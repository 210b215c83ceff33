"""GPU parity of the gated feed-forward block, forward and backward, against its formulas in 64 bits.

Tolerances, as norms of the difference over norms of the result.  Each rounding to bf16 is off by at most 2⁻⁸ of a value
(uniformly spread within that: 2⁻⁸/√3 in norm), and roundings of a product's operands are independent, so they add in
squares:
  h      one rounding of act(g)∘u, both from float32 sums
  y      h's and its own
  dgu    of g and u (they enter act, act' and the products: at most 2 of them in dg, with act' and act at most 1.13 and
         1.2 times as steep as their arguments) and its own
  dx, dW the operands' (dgu or h) and, in bf16, their own
so no norm is off by more than 2⁻⁸·√(1 + 2·1.2² + 1)/√3 = 5.0e-3; float32 sums of K terms add K·2⁻²⁴ at most."""
import math

import pytest
import torch

from tests.gpu_util import empty

pytestmark = pytest.mark.gpu

xt = pytest.importorskip("transformer_fwd_bwd_gb300.xt")

B16 = torch.bfloat16
NORM = 5.0e-3
HALF = 2.0 ** -8


def make(T, d, F, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return n(T, d).to(B16), (n(d, 2 * F) * d ** -0.5).to(B16), (n(F, d) * F ** -0.5).to(B16), n(T, d).to(B16)


def act64(g, act):
    if act == 0:
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    c = torch.special.ndtr(g)
    return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def reference(x, wu, wd, dy, act):
    x, wu, wd, dy = (t.double() for t in (x, wu, wd, dy))
    F = wd.shape[0]
    gu = x @ wu
    g, u = gu[:, :F], gu[:, F:]
    a, da = act64(g, act)
    h = a * u
    dh = dy @ wd.T
    dgu = torch.cat((dh * u * da, dh * a), 1)
    return dict(gu=gu, h=h, y=h @ wd, dgu=dgu, dx=dgu @ wu.T, dw_up=x.T @ dgu, dw_down=h.T @ dy)


def close(got, want, tol=NORM):
    e = float((got.double() - want).norm() / want.norm().clamp(min=1e-300))
    assert e <= tol, e


def bufs(T, d, F, grad="bf16"):
    e = lambda *s: empty(s, "bf16", fill=7.0)  # noqa: E731
    return dict(gu=e(T, 2 * F), h=e(T, F), y=e(T, d), dgu=e(T, 2 * F), dx=e(T, d), dw_up=empty((d, 2 * F), grad, fill=7.0),
                dw_down=empty((F, d), grad, fill=7.0))


CASES = [  # T, d, F, act, dtype of the weights' gradients
    (1, 8, 8, 0, "f32"),
    (1, 768, 2048, 0, "bf16"),
    (3, 16, 72, 1, "bf16"),
    (77, 768, 2048, 0, "f32"),
    (128, 64, 128, 1, "f32"),
    (129, 72, 136, 0, "bf16"),
    (300, 264, 1000, 1, "bf16"),
    (1000, 200, 5464, 0, "f32"),
    (2049, 768, 688, 0, "bf16"),
    (4097, 136, 2056, 1, "f32"),
    (8192, 768, 2048, 0, "f32"),
    (5000, 1032, 2504, 1, "bf16"),
    (100, 64, 20488, 0, "bf16"),   # one row of tiles, wide single-CTA ones
    (128, 200, 10248, 1, "f32"),
]


@pytest.mark.parametrize("T,d,F,act,grad", CASES)
def test_forward_and_backward(T, d, F, act, grad):
    x, wu, wd, dy = make(T, d, F)
    o = bufs(T, d, F, grad)
    ws = xt.gated_mlp_workspace(T, d, F)
    xt.xt_gated_mlp_fwd(x, wu, wd, o["gu"], o["h"], o["y"], act=act, ws=ws)
    xt.xt_gated_mlp_bwd(x, wu, wd, o["gu"], o["h"], dy, o["dgu"], o["dx"], o["dw_up"], o["dw_down"], act=act, ws=ws)
    want = reference(x, wu, wd, dy, act)
    # element by element: g and u are float32 sums of d products, rounded once
    sums = x.double().abs() @ wu.double().abs()
    err = (o["gu"].double() - want["gu"]).abs()
    assert (err <= HALF * want["gu"].abs() + (d + 2) * 2.0 ** -24 * sums).all()
    for name in ("h", "y", "dgu", "dx", "dw_up", "dw_down"):
        close(o[name], want[name])
    assert xt.device_errors() == 0
    # the forward without saved projections: the same h, and h alone
    h2, y2, h3 = empty((T, F), "bf16"), empty((T, d), "bf16"), empty((T, F), "bf16")
    xt.xt_gated_mlp_fwd(x, wu, wd, None, h2, y2, act=act, ws=ws)
    xt.xt_gated_mlp_fwd(x, wu, None, None, h3, None, act=act)
    assert torch.equal(h2, o["h"]) and torch.equal(y2, o["y"]) and torch.equal(h3, o["h"])
    # again: the same bits
    p = bufs(T, d, F, grad)
    xt.xt_gated_mlp_bwd(x, wu, wd, o["gu"], o["h"], dy, p["dgu"], p["dx"], p["dw_up"], p["dw_down"], act=act, ws=ws)
    assert all(torch.equal(p[n], o[n]) for n in ("dgu", "dx", "dw_up", "dw_down"))


def test_accumulation_and_single_gradients():
    T, d, F = 500, 136, 264
    x, wu, wd, dy = make(T, d, F, 3)
    o = bufs(T, d, F, "f32")
    xt.xt_gated_mlp_fwd(x, wu, wd, o["gu"], o["h"], o["y"])
    want = reference(x, wu, wd, dy, 0)
    base = {n: torch.randn_like(o[n].float()).to(o[n].dtype) for n in ("dx", "dw_up", "dw_down")}
    for n in base:
        o[n].copy_(base[n])
    xt.xt_gated_mlp_bwd(x, wu, wd, o["gu"], o["h"], dy, o["dgu"], o["dx"], o["dw_up"], o["dw_down"], acc_dx=1, acc_dw=1)
    for n in base:
        close(o[n], want[n] + base[n].double())
    for n in ("dx", "dw_up", "dw_down"):
        p = bufs(T, d, F, "f32")
        args = {k: (p[k] if k == n else None) for k in ("dx", "dw_up", "dw_down")}
        xt.xt_gated_mlp_bwd(x, wu, wd, o["gu"], o["h"], dy, p["dgu"], args["dx"], args["dw_up"], args["dw_down"])
        close(p[n], want[n])


def test_gradient_against_differences():
    """The formulas in 64 bits that the kernels are held to, against central differences of the forward's."""
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
    x, wu, wd, dy = n(3, 4), n(4, 10), n(5, 4), n(3, 4)
    for act in (0, 1):
        want = reference(x, wu, wd, dy, act)
        for name, t, key in (("x", x, "dx"), ("wu", wu, "dw_up"), ("wd", wd, "dw_down")):
            flat = t.view(-1)
            for i in range(0, flat.numel(), 3):
                keep = float(flat[i])
                vals = []
                for e in (1e-5, -1e-5):
                    flat[i] = keep + e
                    vals.append(float((reference(x, wu, wd, dy, act)["y"] * dy).sum()))
                flat[i] = keep
                assert abs((vals[0] - vals[1]) / 2e-5 - float(want[key].view(-1)[i])) <= 1e-7


@pytest.mark.parametrize("act", [0, 1])
def test_extreme_gates(act):
    """Large projections of either sign, and rows of nought: finite results, as the formula's limits."""
    T, d, F = 130, 64, 136
    x, wu, wd, dy = make(T, d, F, 4)
    x[0] = 0
    x[1] *= 300.0
    x[2] *= -300.0
    o = bufs(T, d, F, "f32")
    xt.xt_gated_mlp_fwd(x, wu, wd, o["gu"], o["h"], o["y"], act=act)
    xt.xt_gated_mlp_bwd(x, wu, wd, o["gu"], o["h"], dy, o["dgu"], o["dx"], o["dw_up"], o["dw_down"], act=act)
    want = reference(x, wu, wd, dy, act)
    assert (o["h"][0] == 0).all() and (o["y"][0] == 0).all()
    for r in (1, 2, 3):
        close(o["h"][r], want["h"][r])
        close(o["dgu"][r], want["dgu"][r], tol=2e-2)  # act' of a rounded g near its steep part: one row of it
    close(o["dx"], want["dx"])


def test_a_row_that_is_not_finite_stays_by_itself():
    T, d, F = 300, 64, 128
    x, wu, wd, dy = make(T, d, F, 5)
    clean = bufs(T, d, F)
    xt.xt_gated_mlp_fwd(x, wu, wd, clean["gu"], clean["h"], clean["y"])
    x[131] = float("nan")
    o = bufs(T, d, F)
    xt.xt_gated_mlp_fwd(x, wu, wd, o["gu"], o["h"], o["y"])
    rest = torch.arange(T, device="cuda") != 131
    assert torch.isnan(o["y"][131]).all() and torch.equal(o["y"][rest], clean["y"][rest])


def test_no_tokens():
    d, F = 64, 128
    x, wu, wd, dy = make(0, d, F)
    e = lambda *s: torch.empty(*s, dtype=B16, device="cuda")  # noqa: E731
    xt.xt_gated_mlp_fwd(x, wu, wd, e(0, 2 * F), e(0, F), e(0, d))
    dw_up, dw_down = empty((d, 2 * F), fill=3.0), empty((F, d), fill=3.0)
    xt.xt_gated_mlp_bwd(x, wu, wd, e(0, 2 * F), e(0, F), dy, e(0, 2 * F), e(0, d), dw_up, dw_down, acc_dw=1)
    assert (dw_up == 3.0).all() and (dw_down == 3.0).all()
    xt.xt_gated_mlp_bwd(x, wu, wd, e(0, 2 * F), e(0, F), dy, e(0, 2 * F), e(0, d), dw_up, dw_down)
    assert (dw_up == 0).all() and (dw_down == 0).all()


def test_streams_and_graphs():
    T, d, F = 900, 200, 520
    sets = [make(T, d, F, s) for s in (1, 2)]

    def go(t, o, ws, s=None):
        xt.xt_gated_mlp_fwd(t[0], t[1], t[2], o["gu"], o["h"], o["y"], ws=ws, s=s)
        xt.xt_gated_mlp_bwd(t[0], t[1], t[2], o["gu"], o["h"], t[3], o["dgu"], o["dx"], o["dw_up"], o["dw_down"], ws=ws, s=s)
    wss = [xt.gated_mlp_workspace(T, d, F) for _ in sets]
    want = [bufs(T, d, F) for _ in sets]
    for t, o, ws in zip(sets, want, wss):
        go(t, o, ws)
    torch.cuda.synchronize()
    got = [bufs(T, d, F) for _ in sets]
    side = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        for t, o, ws, st in zip(sets, got, wss, side):
            go(t, o, ws, st)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(a[n], b[n]) for n in a)
    t = [v.clone() for v in sets[0]]
    o = bufs(T, d, F)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(t, o, wss[0])
    for v, w in zip(t, sets[1]):
        v.copy_(w)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o[n], want[1][n]) for n in o)
