"""Arguments that the operators of packed-document training refuse, on the host: every refusal comes before
anything touches a device."""
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


def rope(xt, x=16, ld_x=64, y=32, ld_y=64, pos=16, axes=2, sections=(8, 24), per_axis=0, base=1e4, T=4, H=1, hd=64, dt=0,
         acc=None):
    sec = (C.c_int32 * max(1, len(sections)))(*sections) if sections is not None else None
    args = [x, ld_x, y, ld_y, pos, axes, sec, per_axis, C.c_double(base), T, H, hd, dt]
    if acc is None:
        return xt.lib().xt_rope_axes_fwd(*args, None)
    return xt.lib().xt_rope_axes_bwd(*args, acc, None)


def test_rope_axes_refusals(xt):
    bad = xt.XT_ERR_INVALID_ARG
    assert rope(xt, dt=2) == bad
    assert rope(xt, hd=63) == bad
    assert rope(xt, hd=258, ld_x=258, ld_y=258, sections=(64, 65)) == xt.XT_ERR_UNSUPPORTED
    assert rope(xt, axes=0) == bad and rope(xt, axes=5, sections=(8, 8, 8, 4, 4)) == bad
    assert rope(xt, sections=(8, 23)) == bad and b"add up" in xt.lib().xt_last_error()
    assert rope(xt, sections=(-8, 40)) == bad
    assert rope(xt, sections=None) == bad
    assert rope(xt, base=0.0) == bad and rope(xt, base=float("nan")) == bad
    assert rope(xt, per_axis=2) == bad
    assert rope(xt, ld_x=63) == bad and rope(xt, ld_y=63) == bad
    assert rope(xt, T=-1) == bad and rope(xt, H=0) == bad
    assert rope(xt, x=None) == bad and rope(xt, y=None) == bad and rope(xt, pos=None) == bad
    assert rope(xt, x=16, y=16, ld_x=64, ld_y=128) == bad
    assert rope(xt, acc=2) == bad and rope(xt, acc=1, x=16, y=16) == bad
    assert rope(xt, T=0, x=None, y=None, pos=None) == xt.XT_OK
    with pytest.raises(ValueError):   # positions of another shape
        xt.xt_rope_axes_fwd(torch.zeros(4, 64), torch.zeros(4, 64), torch.zeros(1, 4, dtype=torch.int32), [8, 24], 1, 64)
    with pytest.raises(ValueError):   # not on a GPU
        xt.xt_rope_axes_fwd(torch.zeros(4, 64), torch.zeros(4, 64), torch.zeros(2, 4, dtype=torch.int32), [8, 24], 1, 64)


def adamw8(xt, n=1, numel=(1000,), ws=8, ws_bytes=1 << 20, shadow_dtype=0, null=None, **kw):
    cfg = xt.adamw_config(**{**dict(lr=1e-3, max_grad_norm=1.0), **kw})
    N = (C.c_int64 * max(1, len(numel)))(*numel)
    lists = [(C.c_void_p * max(1, len(numel)))(*([16] * len(numel))) for _ in range(7)]
    if null is not None:
        lists[null][0] = None
    return xt.lib().xt_adamw8_step(C.byref(cfg), n, *lists[:6], lists[6], shadow_dtype, N, None, ws, ws_bytes, None)


def test_adamw8_refusals(xt):
    bad = xt.XT_ERR_INVALID_ARG
    L = xt.lib()
    assert L.xt_adamw8_step(None, 0, *[None] * 7, 0, None, None, None, 0, None) == bad
    assert adamw8(xt, n=-1) == bad
    assert adamw8(xt, numel=(-5,)) == bad
    assert adamw8(xt, step=0) == bad
    assert adamw8(xt, beta1=1.0) == bad and adamw8(xt, beta2=-0.1) == bad
    assert adamw8(xt, eps=0.0) == bad and adamw8(xt, lr=-1.0) == bad and adamw8(xt, weight_decay=-1.0) == bad
    assert adamw8(xt, shadow_dtype=3) == bad
    for i in range(6):
        assert adamw8(xt, null=i) == bad
    assert adamw8(xt, ws=None) == bad and adamw8(xt, ws_bytes=4) == bad
    assert adamw8(xt, ws=12) == xt.XT_ERR_ALIGNMENT
    assert adamw8(xt, n=0, numel=()) == xt.XT_OK
    n = C.c_int64(0)
    assert [L.xt_adamw8_scales(k, C.byref(n)) or n.value for k in (0, 1, 256, 257)] == [0, 1, 1, 2]
    assert L.xt_adamw8_scales(-1, C.byref(n)) == bad
    assert L.xt_adamw8_workspace_size(1, None, C.byref(C.c_size_t())) == bad
    assert L.xt_adamw8_decode(1, None, None, None, None, None, None, (C.c_int64 * 1)(4), None) == bad
    with pytest.raises(ValueError):   # lists of different lengths
        xt.xt_adamw8_step(xt.adamw_config(1e-3), [], [torch.zeros(1)], [], [], [], [])
    with pytest.raises(ValueError):   # not on a GPU
        xt.xt_adamw8_step(xt.adamw_config(1e-3), [torch.zeros(1)], [torch.zeros(1)], [], [], [], [])


def masked(xt, T=256, H=2, Hkv=1, hd=64, dtype=1, scale=0.0, cap=0.0, plan=16, plan_bytes=1 << 20, q=16, ld_q=128,
           ld_k=64, o=16, lse=16, bwd=False, ws=16, ws_bytes=1 << 20, dk=16, ld_dk=64):
    d = xt.AttentionDesc(T, H, Hkv, hd, dtype, scale, cap, None)
    L = xt.lib()
    if bwd:
        return L.xt_attention_masked_bwd(C.byref(d), plan, plan_bytes, q, ld_q, 16, ld_k, 16, ld_k, o, 128, 16, 128,
                                         lse, 16, 128, dk, ld_dk, 16, 64, ws, ws_bytes, None)
    return L.xt_attention_masked_fwd(C.byref(d), plan, plan_bytes, q, ld_q, 16, ld_k, 16, ld_k, o, 128, lse, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_masked_attention_refusals(xt, bwd):
    bad, uns, ali = xt.XT_ERR_INVALID_ARG, xt.XT_ERR_UNSUPPORTED, xt.XT_ERR_ALIGNMENT
    go = lambda **kw: masked(xt, bwd=bwd, **kw)  # noqa: E731
    assert go(T=-1) == bad and go(T=1 << 30) == bad
    assert go(H=0) == bad and go(H=3, Hkv=2) == bad and go(Hkv=0) == bad
    assert go(dtype=0) == uns
    assert go(hd=32) == uns and go(hd=96) == uns
    assert go(scale=-1.0) == bad and go(scale=float("nan")) == bad
    assert go(cap=-1.0) == bad and go(cap=float("inf")) == bad
    # caps beyond what one exponential resolves, and so small that the scores' multiplier overflows
    assert go(cap=1025.0) == bad and go(cap=1e-40) == bad and go(cap=1e-6, scale=1e34) == bad
    assert go(plan=None) == bad and go(plan=8) == ali and go(plan_bytes=100) == bad
    assert go(q=None) == bad and go(q=24) == ali and go(ld_q=120) == bad and go(ld_q=132) == ali
    assert go(ld_k=56) == bad and go(o=None) == bad and go(lse=None) == bad
    assert go(T=0, plan=None, lse=None, q=None, o=None) == xt.XT_OK
    if bwd:
        assert go(ws=None) == bad and go(ws=8) == ali and go(ws_bytes=100) == bad
        assert go(dk=None) == bad and go(ld_dk=60) == bad and go(ld_dk=68) == ali


def test_attention_plan_refusals(xt):
    bad = xt.XT_ERR_INVALID_ARG
    L = xt.lib()
    n = C.c_size_t(0)
    assert L.xt_attention_plan_size(-1, C.byref(n)) == bad and L.xt_attention_plan_size(1 << 30, C.byref(n)) == bad
    assert L.xt_attention_plan_size(1000, C.byref(n)) == xt.XT_OK
    go = lambda T=1000, docs=4, off=None, causal=1, plan=16, size=n.value: L.xt_attention_plan(  # noqa: E731
        T, docs, off, None, None, causal, plan, size, None)
    assert go(T=-1) == bad and go(T=1 << 30) == bad and go(docs=-1) == bad and go(docs=1 << 30, off=16) == bad
    assert go(docs=3) == bad and go(docs=0) == bad     # equal spans need a divisor
    assert go(causal=2) == bad and go(plan=None) == bad and go(size=n.value - 1) == bad
    assert go(plan=8) == xt.XT_ERR_ALIGNMENT
    assert go(T=0, docs=0, size=64) == xt.XT_OK
    with pytest.raises(ValueError):   # one length per document
        xt.xt_attention_plan(torch.zeros(4), 8, 2, doc_len=torch.zeros(3, dtype=torch.int32))
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    for bad_args in (dict(o=z(4, 64)), dict(k=z(4, 64).float()), dict(v=z(5, 64)), dict(lse=torch.zeros(2, 3)),
                     dict(slopes=torch.zeros(3)), dict(q=z(128, 4).t())):
        a = dict(q=z(4, 128), k=z(4, 64), v=z(4, 64), o=z(4, 128), lse=torch.zeros(2, 4), slopes=None) | bad_args
        with pytest.raises(ValueError):
            xt.xt_attention_masked_fwd(a["q"], a["k"], a["v"], a["o"], a["lse"], z(64), 2, 1, 64, slopes=a["slopes"])
