"""GPU parity of the Muon step against its formulas in 64 bits.

Tolerances.  M and U are a few float32 operations: 3·2⁻²⁴ of the terms' magnitudes.  X: what the operands hold is off by
at most 2⁻²² of their entries and a product's float32 sums by as much again, 2⁻²¹ in all; an error of X grows by at most
a = 3.4445 per step that is left and X itself by no more, so each of the 15 roundings reaches the result as at most
a⁵·2⁻²¹ = 2.3e-4 of ‖X₀‖_F = 1; they are independent and add in squares: ‖X − X*‖_F ≤ √15·485·2⁻²¹ = 9e-4.  (Operands in
one f16 term would be a thousand times further off.)"""
import math

import pytest
import torch

from tests.gpu_util import empty

pytestmark = pytest.mark.gpu

xt = pytest.importorskip("transformer_fwd_bwd_gb300.xt")

EPS = 2.0 ** -24
X_TOL = 9.0e-4
ABC = (3.4445, -4.7750, 2.0315)


def matrices(shapes, seed, size=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    out = []
    for r, c in shapes:
        k = min(8, r, c)
        out.append(size * (n(r, k) @ n(k, c) / math.sqrt(k) + 0.3 * n(r, c)))
    return out


def guarded(ts):
    """Copies between guard bands."""
    out = []
    for t in ts:
        e = empty(tuple(t.shape))
        e.copy_(t)
        out.append(e)
    return out


def reference(g, m, cfg):
    """New momentum and X in 64 bits."""
    f = lambda v: float(torch.tensor(v))  # noqa: E731
    G = g.double() * f(cfg["grad_scale"])
    M = f(cfg["momentum"]) * m.double() + G
    U = G + f(cfg["momentum"]) * M if cfg["nesterov"] else M
    X = U / (U.norm() + cfg["eps"])
    if X.shape[0] > X.shape[1]:
        X = X.T
    for _ in range(cfg["steps"]):
        A = X @ X.T
        X = ABC[0] * X + (ABC[1] * A + ABC[2] * (A @ A)) @ X
    return M, (X.T if g.shape[0] > g.shape[1] else X)


def config(**kw):
    c = dict(lr=0.02, momentum=0.95, weight_decay=0.1, rms=0.2, eps=1e-7, grad_scale=0.25, nesterov=1, steps=5)
    c.update(kw)
    return c


def check(shapes, cfg, seed=1, shadow=None, size=1e-3):
    p, g, m = matrices(shapes, seed, 0.02), matrices(shapes, seed + 1, size), matrices(shapes, seed + 2, 2 * size)
    P, G, M = guarded(p), guarded(g), guarded(m)
    sh = None
    if shadow:
        sh = [empty(s, shadow, fill=9.0) for s in shapes]
        if len(sh) > 1:
            sh[0] = None
    xt.xt_muon_step(xt.muon_config(**cfg), P, G, M, shadows=sh)
    for i, s in enumerate(shapes):
        wm, wx = reference(g[i], m[i], cfg)
        mag = g[i].double().abs() * cfg["grad_scale"] + m[i].double().abs()
        assert ((M[i].double() - wm).abs() <= 3 * EPS * mag).all()
        assert torch.equal(G[i], g[i])
        up = cfg["lr"] * cfg["rms"] * math.sqrt(max(s))
        want = p[i].double() * (1 - cfg["lr"] * cfg["weight_decay"]) - up * wx
        err = float((P[i].double() - want).norm())
        # + two float32 roundings of the weights
        tol = up * X_TOL * cfg["steps"] / 5 + 3 * EPS * float(want.norm() + up * wx.norm())
        assert err <= tol, (s, err, tol)
        if sh and sh[i] is not None:
            assert torch.equal(sh[i], P[i].to(sh[i].dtype))
    assert xt.device_errors() == 0


@pytest.mark.parametrize("shape", [(1, 1), (1, 5), (7, 1), (2, 3), (17, 33), (33, 17), (64, 64), (127, 129), (256, 768),
                                   (768, 256), (300, 300), (1000, 129), (129, 1000), (257, 513), (688, 256), (520, 1032)])
def test_one_matrix(shape):
    check([shape], config(), shadow="bf16")


def test_many_shapes_at_once():
    """More shapes than one launch takes, several matrices of some, in mixed order."""
    shapes = [(64, 192), (64, 64), (64, 344), (172, 64)] * 3 + [(i, 40 + i) for i in range(5, 12)] + [(300, 1), (64, 64)]
    check(shapes, config(), shadow="f32")


def test_more_matrices_than_a_table():
    check([(24, 48)] * 150 + [(48, 24)] * 20, config())


def test_wide_tiles():
    """Enough matrices for 256 x 256 tiles, which pairs of CTAs share, in all three products."""
    check([(300, 700)] * 14 + [(769, 264)] * 8 + [(256, 256)] * 5, config(), shadow="bf16")


@pytest.mark.parametrize("kw", [dict(nesterov=0), dict(momentum=0.0), dict(steps=1), dict(steps=2), dict(steps=8),
                                dict(weight_decay=0.0, grad_scale=1.0), dict(lr=0.0)])
def test_settings(kw):
    cfg = config(**kw)
    # more than five steps: what was rounded off is past its growth (slopes at values near 1 are below 1)
    check([(96, 200), (200, 96)], cfg)


@pytest.mark.parametrize("size", [1e-12, 1e-3, 1e6])
def test_gradient_sizes(size):
    check([(64, 96), (96, 40)], config(eps=1e-20), size=size)


def test_strong_and_weak_directions():
    """A gradient of rank one beside noise 10⁻⁴ as strong: the noise's directions are where errors grow."""
    n, m = 192, 320
    g = torch.randn(n, 1, device="cuda") @ torch.randn(1, m, device="cuda") + 1e-4 * torch.randn(n, m, device="cuda")
    p, buf = torch.zeros(n, m, device="cuda"), torch.zeros(n, m, device="cuda")
    cfg = config(lr=1.0, weight_decay=0.0, rms=1.0 / math.sqrt(m), grad_scale=1.0)
    _, wx = reference(g, buf, cfg)
    xt.xt_muon_step(xt.muon_config(**cfg), [p], [g], [buf])
    assert float((p.double() + wx).norm()) <= X_TOL + 3 * EPS * float(wx.norm())


def test_nought_and_not_finite():
    shapes = [(64, 96), (64, 96), (40, 24)]
    p, g, m = matrices(shapes, 1, 0.02), matrices(shapes, 2), [torch.zeros(s, device="cuda") for s in shapes]
    g[0].zero_()
    g[1][3, 5] = float("nan")
    P = guarded(p)
    cfg = config()
    xt.xt_muon_step(xt.muon_config(**cfg), P, g, m)
    assert torch.equal(P[0], (p[0].double() * (1 - float(torch.tensor(0.02)) * float(torch.tensor(0.1)))).float()) or \
        float((P[0] - p[0] * (1 - 0.002)).abs().max()) <= 2 * EPS * float(p[0].abs().max())
    assert torch.isnan(P[1]).all()
    _, wx = reference(g[2], torch.zeros_like(g[2]), cfg)
    up = 0.02 * 0.2 * math.sqrt(40)
    want = p[2].double() * (1 - 0.002) - up * wx
    assert float((P[2].double() - want).norm()) <= up * X_TOL + 3 * EPS * float(want.norm() + up * wx.norm())


def test_unaligned_buffers_and_what_lies_beside_them():
    r, c = 50, 104
    buf = [torch.full((r * c + 9,), 5.0, device="cuda") for _ in range(3)]
    views = [b[off:off + r * c].view(r, c) for b, off in zip(buf, (1, 3, 2))]
    src = [matrices([(r, c)], s, z)[0] for s, z in ((1, 0.02), (2, 1e-3), (3, 1e-3))]
    for v, s in zip(views, src):
        v.copy_(s)
    al = [s.clone() for s in src]
    cfg = xt.muon_config(**config())
    xt.xt_muon_step(cfg, [views[0]], [views[1]], [views[2]])
    xt.xt_muon_step(cfg, [al[0]], [al[1]], [al[2]])
    # the norm's partial sums are added in another order: the last bits of its reciprocal
    assert float((views[0] - al[0]).norm()) <= 1e-6 * float(al[0].norm()) and torch.equal(views[2], al[2])
    for b, off in zip(buf, (1, 3, 2)):
        assert (b[:off] == 5.0).all() and (b[off + r * c:] == 5.0).all()


def test_streams_graphs_and_equal_bits():
    shapes = [(96, 288), (96, 96), (96, 512), (256, 96)] * 2
    cfg = xt.muon_config(**config())
    sets = [[matrices(shapes, s + k, z) for k, z in ((0, 0.02), (1, 1e-3), (2, 2e-3))] for s in (1, 11)]
    copy = lambda st: [[t.clone() for t in lst] for lst in st]  # noqa: E731
    want = [copy(st) for st in sets]
    for w in want:
        xt.xt_muon_step(cfg, *w)
    torch.cuda.synchronize()
    got = [copy(st) for st in sets]
    wss = [xt.muon_workspace(shapes) for _ in sets]
    side = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for g, ws, st in zip(got, wss, side):
        xt.xt_muon_step(cfg, *g, ws=ws, s=st)
    torch.cuda.synchronize()
    same = lambda a, b: all(torch.equal(x, y) for la, lb in zip(a, b) for x, y in zip(la, lb))  # noqa: E731
    assert same(want[0], got[0]) and same(want[1], got[1])
    cap = copy(sets[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xt.xt_muon_step(cfg, *cap, ws=wss[0])
    for lst, src in zip(cap, sets[1]):
        for t, v in zip(lst, src):
            t.copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    assert same(cap, want[1])
