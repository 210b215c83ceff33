"""GPU parity of the tokens' log probabilities, entropies, most probable tokens and their gradient against the
definition in 64 bits.

Tolerances.  S = Σ exp is summed in float32: a thread adds at most V/512 terms in each of its two sums, 16 more
additions join them (2⁻²⁴ each); a term's exponent t is rounded once (2⁻²⁴·|t|, where only |t| up to 32 matters to
the sum) and ex2 is good to 2 ulp (2⁻²²): relative error of S at most tolS = (V/512 + 16 + 32 + 4)·2⁻²⁴.  logp adds
the rounding of scale·log2(e) (2⁻²⁴·|z|) and of the result.  The entropy is ln S − Σ p t: its second sum has terms of
up to |t|·p, with |t| at most the headroom (8 units of log2) above and the row's spread below the base: (8 + the mean
|t|)·tolS.  A gradient p·(A + B·log p) has p off by (3|log p| + 4)·2⁻²⁴ + tolS relative, plus half a step of its type."""
import math

import pytest
import torch

from tests.gpu_util import empty

pytestmark = pytest.mark.gpu

xt = pytest.importorskip("transformer_fwd_bwd_gb300.xt")

TD = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 2.0 ** -24


def make(R, V, dtype, seed, ld=None, spread=2.5, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = V if ld is None else ld
    buf = torch.full((R * ld + offset + 8,), float("nan"), dtype=TD[dtype], device="cuda")
    x = buf[offset:offset + R * ld].view(R, ld)[:, :V]
    x.copy_(spread * torch.randn(R, V, generator=g, device="cuda"))
    tok = torch.randint(0, V, (R,), generator=g, device="cuda").to(torch.int32)
    return x, tok


def forward(x, tok, top, scale=1.0):
    R = x.shape[0]
    logp, H, stats = empty(R, fill=7.0), empty(R, fill=7.0), empty((R, 2), fill=7.0)
    tl, ti = None, None
    if top:
        tl, ti = empty((R, top), fill=7.0), torch.full((R, top), -7, dtype=torch.int32, device="cuda")
    xt.xt_token_logprobs_fwd(x, tok, logp, H, stats, tl, ti, scale=scale)
    return logp, H, stats, tl, ti


def reference(x, tok, top, scale=1.0):
    z = x.double() * scale
    lp = torch.log_softmax(z, 1)
    p = lp.exp()
    H = torch.special.entr(p).sum(1)
    ids = torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :top]
    return lp, p, H, lp.gather(1, tok.long()[:, None])[:, 0], ids


def tol_sum(V):
    return (V / 512 + 52) * EPS


def check_forward(x, tok, top, scale, out):
    logp, H, stats, tl, ti = out
    V = x.shape[1]
    lp, p, Hr, want, ids = reference(x, tok, top, scale)
    zmax = (x.double() * scale).amax(1)
    tolS = tol_sum(V)
    tol = tolS + EPS * (2 * (x.double().gather(1, tok.long()[:, None])[:, 0] * scale - zmax).abs() + want.abs())
    assert ((logp.double() - want).abs() <= tol).all(), float(((logp.double() - want).abs() / tol).max())
    mean_t = torch.where(p > 0, p * (x.double() * scale - zmax[:, None]).abs(), torch.zeros_like(p)).sum(1)
    tolH = tolS * (8 + mean_t / math.log(2)) + EPS * Hr
    assert ((H.double() - Hr).abs() <= tolH).all(), float(((H.double() - Hr).abs() / tolH).max())
    assert torch.equal(stats[:, 0].double(), x.double().amax(1))
    lse = torch.logsumexp(x.double() * scale, 1) - zmax
    assert ((stats[:, 1].double() - lse).abs() <= tolS + EPS * (lse.abs() + 2)).all()
    if top:
        assert torch.equal(ti.long(), ids)
        want_top = lp.gather(1, ids)
        zt = (x.double().gather(1, ids) * scale - zmax[:, None]).abs()
        err = (tl.double() - want_top).abs()
        err = torch.where(torch.isinf(want_top) & (tl.double() == want_top), torch.zeros_like(err), err)
        tolt = tolS + EPS * (2 * torch.nan_to_num(zt, posinf=0.0) + torch.nan_to_num(want_top.abs(), posinf=0.0))
        assert (err <= tolt).all()


CASES = [  # R, V, dtype, top, scale, ld, offset (elements before the first row)
    (1, 1, "f32", 1, 1.0, None, 0),
    (1, 2, "bf16", 2, 1.0, None, 1),
    (5, 7, "bf16", 5, 0.7, None, 3),
    (9, 33, "f32", 32, 1.0, 40, 1),
    (17, 300, "bf16", 32, 1.25, None, 0),
    (3, 1024, "f32", 0, 1.0, None, 0),
    (4, 2047, "bf16", 20, 1.0, 2051, 5),
    (2, 2049, "bf16", 5, 1.0, None, 0),
    (3, 5000, "f32", 8, 2.0, 5003, 2),
    (1, 50257, "bf16", 5, 1.0, None, 0),
    (3, 50257, "bf16", 32, 1.0, None, 7),
    (70, 50304, "bf16", 1, 1.0, None, 0),
    (400, 20011, "f32", 20, 0.7, None, 0),
    (700, 9999, "bf16", 8, 1.0, None, 0),
    # rows between a warp's and a CTA's, few and many
    (1300, 2500, "bf16", 32, 1.0, None, 0),
    (1300, 4001, "f32", 20, 1.0, 4003, 1),
    (1250, 8191, "bf16", 32, 1.25, None, 3),
    (20, 4000, "bf16", 20, 1.0, None, 0),
    (20, 8000, "bf16", 32, 1.0, None, 0),
    (1300, 70, "bf16", 32, 1.0, None, 0),
    # many long rows
    (700, 16385, "bf16", 20, 1.0, None, 0),
    (1400, 16384, "bf16", 0, 1.0, None, 0),
    (460, 20003, "f32", 32, 1.25, 20009, 3),
    (1000, 33001, "bf16", 1, 1.0, 33007, 5),
    (300, 50257, "bf16", 8, 1.0, None, 0),
    (2, 128256, "f32", 20, 1.0, None, 0),
    (5, 128256, "bf16", 20, 1.0, None, 0),
]


@pytest.mark.parametrize("R,V,dtype,top,scale,ld,offset", CASES)
def test_forward(R, V, dtype, top, scale, ld, offset):
    x, tok = make(R, V, dtype, R + V, ld, offset=offset)
    out = forward(x, tok, top, scale)
    check_forward(x, tok, top, scale, out)
    again = forward(x, tok, top, scale)
    for a, b in zip(out, again):
        assert a is None or torch.equal(a, b)
    assert xt.device_errors() == 0


def grads(x, tok, scale, dl, dh, grad, acc=0, into=None, ld_d=None):
    R, V = x.shape
    logp, H, stats, _, _ = forward(x, tok, 0, scale)
    dx = into if into is not None else empty((R, V), grad)
    xt.xt_token_logprobs_bwd(x, tok, stats, H if dh is not None else None, dl, dh, dx, scale=scale, acc=acc)
    return dx


def gradient(x, tok, scale, dl, dh):
    lp, p, H, _, _ = reference(x, tok, 0, scale)
    R, V = x.shape
    plogp = -torch.special.entr(p)
    dl = torch.zeros(R, dtype=torch.float64, device="cuda") if dl is None else dl.double()
    dh = torch.zeros(R, dtype=torch.float64, device="cuda") if dh is None else dh.double()
    g = -p * dl[:, None] - dh[:, None] * (plogp + p * H[:, None])
    mag = p * dl.abs()[:, None] + dh.abs()[:, None] * (plogp.abs() + p * H[:, None])
    r = torch.arange(R, device="cuda")
    g[r, tok.long()] += dl
    rel = (3 * torch.nan_to_num(lp.abs(), posinf=0.0) + 8 + 3 * H[:, None]) * EPS + 12 * tol_sum(V)
    tol = mag * rel
    tol[r, tok.long()] += 4 * EPS * dl.abs()
    return g * scale, tol * scale


@pytest.mark.parametrize("R,V,dtype,grad,scale,ld,offset,which", [
    (1, 1, "f32", "f32", 1.0, None, 0, "both"),
    (6, 9, "bf16", "bf16", 1.0, None, 1, "both"),
    (5, 300, "bf16", "f32", 0.7, 311, 3, "both"),
    (3, 1025, "f32", "bf16", 1.0, None, 1, "logp"),
    (7, 4097, "f32", "f32", 1.25, None, 0, "entropy"),
    (3, 50257, "bf16", "bf16", 1.0, None, 0, "both"),
    (40, 50304, "bf16", "bf16", 1.0, None, 0, "both"),
    (4, 128256, "f32", "f32", 1.0, None, 0, "both"),
])
def test_gradient(R, V, dtype, grad, scale, ld, offset, which):
    x, tok = make(R, V, dtype, 3 * R + V, ld, offset=offset)
    g = torch.Generator(device="cuda").manual_seed(5)
    dl = torch.randn(R, generator=g, device="cuda") if which != "entropy" else None
    dh = torch.randn(R, generator=g, device="cuda") if which != "logp" else None
    want, tol = gradient(x, tok, scale, dl, dh)
    half = 2.0 ** -8 if grad == "bf16" else EPS
    dx = grads(x, tok, scale, dl, dh, grad)
    bound = tol + half * want.abs() + 1e-38
    assert ((dx.double() - want).abs() <= bound).all(), float(((dx.double() - want).abs() / bound).max())
    # accumulation adds to what is there
    base = torch.randn(R, V, generator=g, device="cuda").to(TD[grad])
    acc = empty((R, V), grad)
    acc.copy_(base)
    grads(x, tok, scale, dl, dh, grad, acc=1, into=acc)
    total = want + base.double()
    bound = tol + half * total.abs() + 2 * EPS * (want.abs() + base.double().abs())
    assert ((acc.double() - total).abs() <= bound).all()
    if dtype == grad and ld is None:  # in place: the same bits
        y = x.clone()
        logp, H, stats, _, _ = forward(y, tok, 0, scale)
        xt.xt_token_logprobs_bwd(y, tok, stats, H, dl, dh, y, scale=scale)
        assert torch.equal(y, dx)


def test_gradient_against_differences():
    """The analytic gradient in 64 bits that the kernel is held to, against central differences of the definition."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(3, 11, generator=g, device="cuda", dtype=torch.float64)
    tok = torch.tensor([0, 10, 4], dtype=torch.int32, device="cuda")
    dl, dh = (torch.randn(3, generator=g, device="cuda", dtype=torch.float64) for _ in range(2))

    def value(y):
        lp = torch.log_softmax(y * 1.3, 1)
        return (dl * lp.gather(1, tok.long()[:, None])[:, 0]).sum() + (dh * -(lp.exp() * lp).sum(1)).sum()
    want, _ = gradient(x, tok, 1.3, dl, dh)
    for r in range(3):
        for v in range(11):
            e = torch.zeros_like(x)
            e[r, v] = 1e-5
            # third-order remainder ~1e-10·|f'''|, rounding 1e-16/1e-5
            assert abs(float((value(x + e) - value(x - e)) / 2e-5 - want[r, v])) <= 1e-8
    dx = grads(x.float(), tok, 1.3, dl.float(), dh.float(), "f32")
    w32, tol = gradient(x.float(), tok, 1.3, dl.float(), dh.float())
    assert ((dx.double() - w32).abs() <= tol + EPS * w32.abs()).all()


@pytest.mark.parametrize("V", [257, 2047, 5001, 50257])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("times", [1, 220])
def test_ties_and_order(V, dtype, times):
    """Equal logits by rising id, whichever threads hold them; rows that rise, fall and are constant."""
    rows = [torch.zeros(V), torch.arange(V) // 3, -(torch.arange(V) // 5), (torch.arange(V) * 7919) % 13,
            torch.where(torch.arange(V) % 256 == 3, 1.0, 0.0), torch.tensor([0.0, -0.0]).repeat(V)[:V]]
    # enough copies that other kernels take the rows
    x = torch.stack([r.float() for r in rows]).to(TD[dtype]).cuda().repeat(times if V < 10000 else 1, 1)
    tok = (torch.arange(x.shape[0], device="cuda") % V).to(torch.int32)
    out = forward(x, tok, 32)
    check_forward(x, tok, 32, 1.0, out)


@pytest.mark.parametrize("V,dtype", [(40, "f32"), (3000, "bf16"), (50257, "bf16"), (128256, "f32")])
def test_banned_extreme_and_empty_rows(V, dtype):
    lowest = torch.finfo(TD[dtype]).min
    R = 10
    x, tok = make(R, V, dtype, 11)
    x[0, 5:] = -math.inf                       # five tokens allowed
    tok[0] = 4
    x[1] = lowest                              # the mask leaves nothing: uniform
    x[2, :] = -math.inf                        # no distribution
    x[3, V // 2] = float("nan")
    x[4, 1] = math.inf
    x[5, :] = -math.inf
    x[5, V - 1] = 3.0                          # one token
    tok[5] = V - 1
    x[6, ::2] = lowest
    x[7] = x[7].float().mul(100.0).add(20000.0).to(TD[dtype])  # far from nought
    x[8, 0] = 1000.0                           # one far above the rest
    x[9] = lowest
    x[9, 3] = 0.9 * lowest
    top = min(20, V)
    logp, H, stats, tl, ti = forward(x, tok, top)
    bad = [2, 3, 4]
    good = [0, 1, 5, 6, 7, 8, 9]
    for t in (logp, H, stats, tl):
        assert torch.isnan(t[bad]).all()
    assert (ti[bad] == -1).all()
    lp, p, Hr, want, ids = reference(x[good], tok[good], top)
    tolS = tol_sum(V)
    assert torch.equal(ti[good].long(), ids)
    same = (logp[good].double() == want) | ((logp[good].double() - want).abs() <= tolS + 4 * EPS * (want.abs() + 1))
    assert same.all()
    assert ((H[good].double() - Hr).abs() <= 40 * tolS).all()
    wt = lp.gather(1, ids)
    assert ((tl[good].double() == wt) | ((tl[good].double() - wt).abs() <= tolS + 4 * EPS * (wt.abs() + 1))).all()
    assert xt.device_errors() == 0
    # gradients: banned tokens have none, bad rows NaN unless nothing comes from above
    g = torch.Generator(device="cuda").manual_seed(2)
    dl, dh = torch.randn(R, generator=g, device="cuda"), torch.randn(R, generator=g, device="cuda")
    dl[3] = dh[3] = 0.0
    dx = empty((R, V))
    xt.xt_token_logprobs_bwd(x, tok, stats, H, dl, dh, dx)
    assert torch.isnan(dx[[2, 4]]).all() and (dx[3] == 0).all()
    gw, gt = gradient(x[good], tok[good], 1.0, dl[good], dh[good])
    # float32 holds no more than 2^-126 of p: smaller ones come out as 0
    bound = gt + EPS * gw.abs() + 40 * tolS * (gw.abs()) + 1e-36
    # a row far from nought: its exponent is formed from the difference to the maximum, no further error
    assert ((dx[good].double() - gw).abs() <= bound).all()
    assert (dx[0, 5:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_long_rows_of_every_kind(dtype):
    """Many long rows, the odd ones among them: ties, rising, banned, empty, not finite; each row equal to the same row on
    its own (which a cluster of CTAs takes) up to the sums' order."""
    V, n = 17000, 500
    x, tok = make(n, V, dtype, 21)
    x[3] = 0.0
    x[4] = (torch.arange(V, device="cuda") // 3).to(TD[dtype])
    x[5, ::2] = -math.inf
    x[6] = -math.inf
    x[7, 99] = float("nan")
    x[8, 100] = math.inf
    x[9] = torch.finfo(TD[dtype]).min
    x[10, 7] = 500.0
    tok[5] = 1
    out = forward(x, tok, 20)
    for r in range(12):
        one = forward(x[r:r + 1], tok[r:r + 1], 20)
        assert torch.equal(out[4][r:r + 1], one[4])
        for a, b in zip(out[:4], one[:4]):
            both = torch.isnan(a[r:r + 1]) & torch.isnan(b) | (a[r:r + 1] == b)
            assert (both | ((a[r:r + 1] - b).abs() <= 40 * tol_sum(V) + 4 * EPS * b.abs())).all()
    good = [r for r in range(n) if r not in (5, 6, 7, 8, 9)]
    check_forward(x[good], tok[good], 20, 1.0, tuple(o[good] for o in out))
    assert xt.device_errors() == 0


def test_tokens_outside_the_vocabulary():
    x, tok = make(4, 600, "f32", 1)
    tok[1], tok[2] = -1, 600
    xt.clear_device_errors()
    logp, H, stats, tl, ti = forward(x, tok, 3)
    assert torch.isnan(logp[[1, 2]]).all() and torch.isfinite(logp[[0, 3]]).all()
    assert torch.isfinite(H).all() and (ti >= 0).all()
    assert xt.device_errors() == xt.XT_DEVERR_INDEX
    xt.clear_device_errors()
    dl = torch.tensor([1.0, 1.0, 0.0, 1.0], device="cuda")
    dx = empty((4, 600))
    xt.xt_token_logprobs_bwd(x, tok, stats, None, dl, None, dx)
    assert torch.isnan(dx[1]).all() and (dx[2] == 0).all() and torch.isfinite(dx[[0, 3]]).all()
    assert xt.device_errors() == xt.XT_DEVERR_INDEX
    xt.clear_device_errors()


def test_strided_rows_leave_the_rest_alone_and_long_offsets():
    x, tok = make(5, 300, "bf16", 3, ld=320)
    buf = torch.full((5, 320), 9.0, dtype=torch.bfloat16, device="cuda")
    dl = torch.ones(5, device="cuda")
    logp, H, stats, _, _ = forward(x, tok, 0)
    xt.xt_token_logprobs_bwd(x, tok, stats, H, dl, dl, buf[:, :300])
    assert (buf[:, 300:] == 9.0).all()
    want, tol = gradient(x, tok, 1.0, dl, dl)
    assert ((buf[:, :300].double() - want).abs() <= tol + 2.0 ** -8 * want.abs() + 1e-38).all()
    # rows whose offset passes 2^31 elements
    big = torch.empty(45000, 50304, dtype=torch.bfloat16, device="cuda")
    big[-2:] = make(2, 50304, "bf16", 4)[0]
    ld, last = 50304, big[-2:]
    assert (45000 - 2) * ld > 2 ** 31
    whole = torch.randint(0, ld, (45000,), device="cuda").to(torch.int32)
    lp = torch.empty(45000, device="cuda")
    big[:-2] = 0.0
    ti, tl = torch.empty(45000, 4, dtype=torch.int32, device="cuda"), torch.empty(45000, 4, device="cuda")
    st, ent = torch.empty(45000, 2, device="cuda"), torch.empty(45000, device="cuda")
    xt.xt_token_logprobs_fwd(big, whole, lp, ent, st, tl, ti)
    check_forward(last, whole[-2:], 4, 1.0, (lp[-2:], ent[-2:], st[-2:], tl[-2:], ti[-2:]))
    ones = torch.ones(45000, device="cuda")
    xt.xt_token_logprobs_bwd(big, whole, st, ent, ones, ones, big)
    want, tol = gradient(make(2, 50304, "bf16", 4)[0], whole[-2:], 1.0, ones[-2:], ones[-2:])
    assert ((big[-2:].double() - want).abs() <= tol + 2.0 ** -8 * want.abs() + 1e-38).all()


def test_streams_and_graphs():
    """Two streams at once, and a captured pair replayed on new logits."""
    xs = [make(33, 7001, "bf16", s) for s in (1, 2)]
    want = [forward(x, t, 8) for x, t in xs]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in xs]
    got = [tuple(torch.empty_like(o) for o in w) for w in want]
    for (x, t), st, o in zip(xs, side, got):
        for _ in range(3):
            xt.xt_token_logprobs_fwd(x, t, *o, s=st)
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, o))
    x, t = xs[0][0].clone(), xs[0][1].clone()
    o = got[0]
    dl, dx = torch.ones(33, device="cuda"), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xt.xt_token_logprobs_fwd(x, t, *o)
        xt.xt_token_logprobs_bwd(x, t, o[2], o[1], dl, dl, dx)
    x.copy_(xs[1][0])
    t.copy_(xs[1][1])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[1], o))
    assert torch.equal(dx, grads(x, t, 1.0, dl, dl, "bf16"))
