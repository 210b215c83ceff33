"""GPU parity of the scaled embedding lookup and its gradient by sorted tokens against 64-bit sums.

Tolerances.  h is one float32 product of exact inputs (2⁻²⁴) and one rounding to its type.  A gradient's row adds its n
tokens' rows in float32: at most n·2⁻²⁴ of the sum of magnitudes, plus the product with the scale and the addition to
what was there (2⁻²⁴ each) and half a step of its type."""
import numpy as np
import pytest
import torch

from tests.gpu_util import empty

pytestmark = pytest.mark.gpu

xt = pytest.importorskip("transformer_fwd_bwd_gb300.xt")

TD = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 2.0 ** -24


def half(dtype):
    return 2.0 ** -8 if dtype == "bf16" else EPS


def draw_ids(kind, T, V, seed):
    r = np.random.default_rng(seed)
    if kind == "uniform":
        a = r.integers(0, V, T)
    elif kind == "one":
        a = np.full(T, V - 1)
    elif kind == "two":
        a = r.choice([0, V // 2], T)
    elif kind == "rising":
        a = np.arange(T) % V
    elif kind == "pad":  # most of them padding
        a = np.where(r.random(T) < 0.8, 3, r.integers(0, V, T))
    else:  # falling frequencies
        w = 1.0 / (np.arange(V) + 10.0)
        a = r.choice(V, T, p=w / w.sum())
    return torch.tensor(a.astype(np.int32), device="cuda")


def rows(T, d, dtype, seed, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.empty(T * d + offset, dtype=TD[dtype], device="cuda")
    x = buf[offset:].view(T, d)
    x.copy_(torch.randn(T, d, generator=g, device="cuda"))
    return x


def want_grad(ids, dh, V, scale, base=None):
    d = dh.shape[1]
    s, m = torch.zeros(V, d, dtype=torch.float64, device="cuda"), torch.zeros(V, d, dtype=torch.float64, device="cuda")
    ok = (ids >= 0) & (ids < V)
    s.index_add_(0, ids[ok].long(), dh[ok].double())
    m.index_add_(0, ids[ok].long(), dh[ok].double().abs())
    n = torch.bincount(ids[ok].long(), minlength=V).double()[:, None]
    want = s * scale
    tol = (n + 2) * EPS * m * abs(scale)
    if base is not None:
        want, tol = want + base.double(), tol + EPS * (want.abs() + base.double().abs())
    return want, tol


def check_plan(plan, ids, V):
    T = ids.numel()
    e = plan[16:16 + 8 * T].view(torch.int64)
    key = torch.where((ids >= 0) & (ids < V), ids, torch.full_like(ids, V)).long()
    order = torch.sort(key, stable=True).indices
    assert torch.equal(e & 0xFFFFFFFF, order) and torch.equal(e >> 32, key[order])


CASES = [  # T, d, V, dtype of dh, of dE, ids, elements before the first row
    (1, 1, 1, "f32", "f32", "one", 0),
    (1, 768, 50304, "bf16", "f32", "uniform", 0),
    (2, 8, 300, "bf16", "bf16", "one", 0),
    (37, 768, 50304, "bf16", "f32", "falling", 0),
    (33, 17, 511, "f32", "bf16", "uniform", 0),
    (255, 264, 512, "bf16", "f32", "two", 0),
    (1025, 40, 513, "f32", "f32", "rising", 0),
    (3000, 256, 262143, "bf16", "f32", "uniform", 0),
    (4097, 300, 262144, "bf16", "bf16", "falling", 2),
    (8192, 768, 50304, "bf16", "f32", "falling", 0),
    (8192, 64, 50304, "f32", "f32", "one", 0),
    (9001, 520, 1000, "bf16", "f32", "pad", 0),
    (40000, 48, 128256, "bf16", "f32", "pad", 0),
    (70001, 129, 7, "f32", "f32", "uniform", 1),
]


@pytest.mark.parametrize("T,d,V,dtype,grad,kind,offset", CASES)
@pytest.mark.parametrize("acc", [0, 1])
def test_gradient(T, d, V, dtype, grad, kind, offset, acc):
    ids, dh = draw_ids(kind, T, V, T + d), rows(T, d, dtype, T, offset)
    scale = float(d) ** 0.5
    plan = xt.embedding_plan_buffer(T)
    xt.xt_embedding_plan(ids, V, plan)
    check_plan(plan, ids, V)
    base = rows(V, d, grad, 5)
    dE = empty((V, d), grad)
    dE.copy_(base)
    xt.xt_embedding_sorted_bwd(plan, dh, dE, scale=scale, acc=acc)
    want, tol = want_grad(ids, dh, V, scale, base if acc else None)
    bound = tol + half(grad) * want.abs()
    err = (dE.double() - want).abs()
    assert (err <= bound).all(), float((err / (bound + 1e-300)).max())
    again = base.clone()
    xt.xt_embedding_sorted_bwd(plan, dh, again, scale=scale, acc=acc)
    assert torch.equal(again, dE)
    assert xt.device_errors() == 0


@pytest.mark.parametrize("T,d,dt_e,dt_h,scale", [(1, 1, "f32", "f32", 1.0), (5, 24, "bf16", "bf16", 1.0),
                                                 (700, 768, "bf16", "bf16", 27.7), (33, 17, "f32", "bf16", -2.0),
                                                 (100, 8, "bf16", "f32", 0.5), (9000, 520, "f32", "f32", 1.5)])
def test_lookup(T, d, dt_e, dt_h, scale):
    V = 999
    E, ids = rows(V, d, dt_e, 1), draw_ids("uniform", T, V, 2)
    h = empty((T, d), dt_h)
    xt.xt_embedding_lookup_fwd(ids, E, h, scale=scale)
    s = float(torch.tensor(scale))
    want = E.double()[ids.long()] * s
    assert ((h.double() - want).abs() <= (EPS + half(dt_h)) * want.abs()).all()
    if scale == 1.0 and dt_e == dt_h:
        assert torch.equal(h, E[ids.long()])


def test_ids_outside_the_vocabulary_and_no_tokens():
    V, d = 50, 40
    ids = torch.tensor([3, -1, 3, 50, 49, 2 ** 31 - 1, -2 ** 31, 0], dtype=torch.int32, device="cuda")
    E, dh = rows(V, d, "f32", 1), rows(8, d, "f32", 2)
    xt.clear_device_errors()
    h = empty((8, d))
    xt.xt_embedding_lookup_fwd(ids, E, h)
    bad = torch.tensor([1, 3, 5, 6], device="cuda")
    assert torch.isnan(h[bad]).all() and torch.equal(h[[0, 2, 4, 7]], E[[3, 3, 49, 0]])
    assert xt.device_errors() == xt.XT_DEVERR_INDEX
    xt.clear_device_errors()
    plan = xt.embedding_plan_buffer(8)
    xt.xt_embedding_plan(ids, V, plan)
    assert xt.device_errors() == xt.XT_DEVERR_INDEX
    xt.clear_device_errors()
    dh[bad] = float("nan")  # left out, whatever it holds
    for acc in (0, 1):
        dE = empty((V, d), fill=1.0)
        xt.xt_embedding_sorted_bwd(plan, dh, dE, acc=acc)
        clean = dh.clone()
        clean[bad] = 0
        want, tol = want_grad(ids, clean, V, 1.0, torch.ones(V, d, device="cuda") if acc else None)
        assert ((dE.double() - want).abs() <= tol + EPS * want.abs()).all()
    # many bad ids: they cross chunks
    ids = torch.full((300,), -5, dtype=torch.int32, device="cuda")
    ids[:40] = 7
    plan = xt.embedding_plan_buffer(300)
    xt.xt_embedding_plan(ids, V, plan)
    dh = rows(300, d, "f32", 3)
    dE = empty((V, d), fill=2.0)
    xt.xt_embedding_sorted_bwd(plan, dh, dE)
    want, tol = want_grad(ids, dh, V, 1.0)
    assert ((dE.double() - want).abs() <= tol + EPS * want.abs()).all()
    xt.clear_device_errors()
    # no tokens
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    plan = xt.embedding_plan_buffer(0)
    xt.xt_embedding_plan(none, V, plan)
    dE = empty((V, d), fill=3.0)
    xt.xt_embedding_sorted_bwd(plan, torch.empty(0, d, device="cuda"), dE, acc=1)
    assert (dE == 3.0).all()
    xt.xt_embedding_sorted_bwd(plan, torch.empty(0, d, device="cuda"), dE, acc=0)
    assert (dE == 0.0).all() and xt.device_errors() == 0


def test_far_rows():
    """A table of more than 2^31 elements, ids of 22 bits (three digits of the sort)."""
    V, d, T = 2200000, 1024, 3000
    E = torch.empty(V, d, dtype=torch.bfloat16, device="cuda")
    ids = draw_ids("uniform", T, V, 4)
    ids[:5] = V - 1
    ids[5] = 0
    E[ids.long()] = rows(T, d, "bf16", 1)
    h = empty((T, d), "bf16")
    xt.xt_embedding_lookup_fwd(ids, E, h)
    assert torch.equal(h, E[ids.long()])
    plan = xt.embedding_plan_buffer(T)
    xt.xt_embedding_plan(ids, V, plan)
    check_plan(plan, ids, V)
    E.fill_(7.0)
    dh = rows(T, d, "bf16", 2)
    xt.xt_embedding_sorted_bwd(plan, dh, E, acc=0)
    used, at = torch.unique(ids.long(), return_inverse=True)
    want = torch.zeros(used.numel(), d, dtype=torch.float64, device="cuda").index_add_(0, at, dh.double())
    mag = torch.zeros_like(want).index_add_(0, at, dh.double().abs())
    assert ((E[used].double() - want).abs() <= 12 * EPS * mag + half("bf16") * want.abs()).all()
    E[used] = 0
    assert not E.any()
    assert xt.device_errors() == 0


def test_plan_of_other_sizes_is_refused():
    V, d = 100, 16
    ids = draw_ids("uniform", 64, V, 1)
    plan = xt.embedding_plan_buffer(64)
    xt.xt_embedding_plan(ids, V, plan)
    xt.clear_device_errors()
    for T, W in ((63, V), (64, V - 1)):
        dE = empty((W, d), fill=5.0)
        xt.xt_embedding_sorted_bwd(plan, rows(T, d, "f32", 1), dE)
        assert (dE == 5.0).all() and xt.device_errors() == xt.XT_DEVERR_PLAN
        xt.clear_device_errors()


def test_one_plan_for_two_tables_on_two_streams_and_in_a_graph():
    T, V = 5000, 3001
    ids = draw_ids("falling", T, V, 1)
    plan = xt.embedding_plan_buffer(T)
    xt.xt_embedding_plan(ids, V, plan)
    dhs = [rows(T, d, "bf16", d) for d in (64, 136)]
    want = []
    for dh in dhs:
        dE = torch.empty(V, dh.shape[1], device="cuda")
        xt.xt_embedding_sorted_bwd(plan, dh, dE, scale=2.0)
        want.append(dE)
    torch.cuda.synchronize()
    got = [torch.full_like(w, 7.0) for w in want]
    wss = [xt.embedding_sorted_workspace(T, dh.shape[1]) for dh in dhs]
    side = [torch.cuda.Stream() for _ in dhs]
    for dh, o, st, ws in zip(dhs, got, side, wss):
        for _ in range(3):
            xt.xt_embedding_sorted_bwd(plan, dh, o, scale=2.0, ws=ws, s=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    new = ids.clone()
    out = torch.empty_like(want[0])
    with torch.cuda.graph(graph):
        xt.xt_embedding_plan(new, V, plan)
        xt.xt_embedding_sorted_bwd(plan, dhs[0], out, scale=2.0, ws=wss[0])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])
    new.copy_(draw_ids("pad", T, V, 9))
    graph.replay()
    torch.cuda.synchronize()
    w, tol = want_grad(new, dhs[0], V, 2.0)
    assert ((out.double() - w).abs() <= tol + EPS * w.abs()).all()
