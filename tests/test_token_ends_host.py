"""Arguments that the token log probabilities and the sorted embedding gradient refuse, on the host: every refusal comes
before anything touches a device."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def xt():
    from transformer_fwd_bwd_gb300 import build
    build.build()
    from transformer_fwd_bwd_gb300 import xt as m
    m.lib()
    return m


def logprobs(xt, x=16, ld=100, tokens=16, scale=1.0, top=0, logp=16, top_logp=16, top_ids=16, rows=4, V=100, dt=0):
    return xt.lib().xt_token_logprobs_fwd(x, ld, tokens, C.c_float(scale), top, logp, None, None, top_logp, top_ids, rows,
                                          V, dt, None)


def logprobs_bwd(xt, x=16, ld=100, tokens=16, stats=16, entropy=16, d_logp=16, d_entropy=16, scale=1.0, dx=32, ld_d=100,
                 rows=4, V=100, dt=0, dt_grad=0, acc=0):
    return xt.lib().xt_token_logprobs_bwd(x, ld, tokens, stats, entropy, d_logp, d_entropy, C.c_float(scale), dx, ld_d,
                                          rows, V, dt, dt_grad, acc, None)


@pytest.mark.parametrize("f", [logprobs, logprobs_bwd])
def test_logprobs_refusals(xt, f):
    bad = xt.XT_ERR_INVALID_ARG
    assert f(xt, dt=2) == bad and f(xt, rows=-1) == bad and f(xt, V=0) == bad and f(xt, V=1 << 30, ld=1 << 30) == bad
    assert f(xt, rows=1 << 31) == bad and f(xt, ld=99) == bad
    for scale in (0.0, -1.0, 1e-7, 1e7, float("nan"), float("inf")):
        assert f(xt, scale=scale) == bad
    assert f(xt, x=None) == bad and f(xt, tokens=None) == bad
    assert f(xt, x=18) == xt.XT_ERR_ALIGNMENT
    assert f(xt, rows=0, x=None, tokens=None) == xt.XT_OK


def test_logprobs_forward_refusals(xt):
    bad = xt.XT_ERR_INVALID_ARG
    assert logprobs(xt, top=-1) == bad and logprobs(xt, top=5, V=4, ld=4) == bad
    assert logprobs(xt, top=33) == xt.XT_ERR_UNSUPPORTED
    assert logprobs(xt, logp=None) == bad and logprobs(xt, top=3, top_ids=None) == bad
    assert logprobs(xt, top=3, top_logp=None) == bad
    z, t = torch.zeros(4, 9), torch.zeros(4, dtype=torch.int32)
    v = torch.zeros(4)
    for args in ((z.t(), t, v), (z, t.long(), v), (z, t[:3], v), (z, t, v.double()), (z, t, v, v[:3]),
                 (z, t, v, v, torch.zeros(4)), (z, t, v, v, None, torch.zeros(4, 2)),
                 (z, t, v, v, None, torch.zeros(4, 2), torch.zeros(4, 2)), (z, t, v)):  # the last: not on a GPU
        with pytest.raises(ValueError):
            xt.xt_token_logprobs_fwd(*args)


def test_logprobs_backward_refusals(xt):
    bad, f = xt.XT_ERR_INVALID_ARG, logprobs_bwd
    assert f(xt, dt_grad=2) == bad and f(xt, ld_d=99) == bad and f(xt, acc=2) == bad
    assert f(xt, stats=None) == bad and f(xt, dx=None) == bad and f(xt, entropy=None) == bad
    assert f(xt, dx=34) == xt.XT_ERR_ALIGNMENT
    # in place: another type, another stride, or adding to what is read
    assert f(xt, dx=16, dt_grad=1) == bad and f(xt, dx=16, ld_d=104) == bad and f(xt, dx=16, acc=1) == bad
    with pytest.raises(ValueError):
        xt.xt_token_logprobs_bwd(torch.zeros(4, 9), torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2), None, None, None,
                                 torch.zeros(4, 8))


def test_embedding_refusals(xt):
    bad, ali, L = xt.XT_ERR_INVALID_ARG, xt.XT_ERR_ALIGNMENT, xt.lib()
    n = C.c_size_t(0)

    def look(ids=16, E=16, h=16, T=4, d=8, V=10, dt_e=0, dt_h=0):
        return L.xt_embedding_lookup_fwd(ids, E, h, T, d, V, C.c_float(1.0), dt_e, dt_h, None)

    assert look(T=-1) == bad and look(T=1 << 30) == bad and look(d=0) == bad and look(V=0) == bad
    assert look(V=(1 << 31) - 1) == bad and look(dt_e=2) == bad and look(dt_h=-1) == bad
    assert look(ids=None) == bad and look(E=None) == bad and look(h=None) == bad
    assert look(T=0, ids=None, E=None, h=None) == xt.XT_OK
    assert L.xt_embedding_plan_size(-1, C.byref(n)) == bad and L.xt_embedding_plan_size(4, None) == bad
    assert L.xt_embedding_plan_size(1000, C.byref(n)) == xt.XT_OK
    size = n.value

    def plan(ids=16, T=1000, V=10, p=16, b=size):
        return L.xt_embedding_plan(ids, T, V, p, b, None)

    assert plan(T=-1) == bad and plan(V=0) == bad and plan(ids=None) == bad and plan(p=None) == bad
    assert plan(b=size - 1) == bad and plan(p=8) == ali
    assert L.xt_embedding_sorted_bwd_workspace_size(-1, 4, C.byref(n)) == bad
    assert L.xt_embedding_sorted_bwd_workspace_size(4, 0, C.byref(n)) == bad
    assert L.xt_embedding_sorted_bwd_workspace_size(1000, 8, C.byref(n)) == xt.XT_OK
    room = n.value

    def grad(p=16, b=size, dh=16, dE=16, T=1000, d=8, V=10, dt=0, dg=0, acc=0, ws=16, wb=room):
        return L.xt_embedding_sorted_bwd(p, b, dh, dE, T, d, V, C.c_float(1.0), dt, dg, acc, ws, wb, None)

    assert grad(p=None) == bad and grad(b=size - 1) == bad and grad(p=8) == ali
    assert grad(dh=None) == bad and grad(dE=None) == bad and grad(dt=2) == bad and grad(dg=2) == bad and grad(acc=2) == bad
    assert grad(ws=None) == bad and grad(wb=room - 1) == bad and grad(ws=8) == ali
    assert grad(d=0) == bad and grad(V=0) == bad and grad(T=-1) == bad
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):   # ids of another type
        xt.xt_embedding_lookup_fwd(i32.long(), torch.zeros(5, 8), torch.zeros(4, 8))
    with pytest.raises(ValueError):   # rows of another number
        xt.xt_embedding_lookup_fwd(i32, torch.zeros(5, 8), torch.zeros(3, 8))
    with pytest.raises(ValueError):
        xt.xt_embedding_plan(i32.long(), 5, torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(ValueError):   # not on a GPU
        xt.xt_embedding_plan(i32, 5, torch.zeros(96, dtype=torch.uint8))
    with pytest.raises(ValueError):   # rows of another width
        xt.xt_embedding_sorted_bwd(torch.zeros(96, dtype=torch.uint8), torch.zeros(4, 7), torch.zeros(5, 8))
