"""Arguments that the Muon step refuses, on the host: every refusal comes before anything touches a device."""
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


def step(xt, shapes=((8, 16),), n=None, ws=16, ws_bytes=1 << 30, shadow_dtype=0, null=None, **kw):
    cfg = xt.muon_config(**{**dict(lr=1e-3), **kw})
    n = len(shapes) if n is None else n
    lists = [(C.c_void_p * max(1, len(shapes)))(*([16] * len(shapes))) for _ in range(4)]
    if null is not None:
        lists[null][0] = None
    R = (C.c_int64 * max(1, len(shapes)))(*[r for r, _ in shapes])
    S = (C.c_int64 * max(1, len(shapes)))(*[c for _, c in shapes])
    return xt.lib().xt_muon_step(C.byref(cfg), n, *lists, shadow_dtype, R, S, ws, ws_bytes, None)


def test_refusals(xt):
    bad, L = xt.XT_ERR_INVALID_ARG, xt.lib()
    assert L.xt_muon_step(None, 0, None, None, None, None, 0, None, None, None, 0, None) == bad
    assert step(xt, n=-1) == bad
    for shape in ((0, 4), (4, 0), (-1, 4), ((1 << 20) + 1, 1), (1 << 16, 1 << 15)):
        assert step(xt, shapes=(shape,)) == bad
    nan, inf = float("nan"), float("inf")
    for kw in (dict(momentum=1.0), dict(momentum=-0.1), dict(momentum=nan), dict(lr=-1.0), dict(lr=inf), dict(lr=nan),
               dict(weight_decay=-1.0), dict(weight_decay=nan), dict(rms=-1.0), dict(rms=inf), dict(eps=0.0), dict(eps=nan),
               dict(grad_scale=nan), dict(grad_scale=inf), dict(steps=0), dict(steps=21), dict(nesterov=2),
               dict(nesterov=-1)):
        assert step(xt, **kw) == bad, kw
    assert step(xt, shadow_dtype=3) == bad
    for i in range(3):
        assert step(xt, null=i) == bad
    assert step(xt, ws=None) == bad and step(xt, ws_bytes=64) == bad and step(xt, ws=24) == xt.XT_ERR_ALIGNMENT
    assert step(xt, shapes=[(4, i + 1) for i in range(65)]) == xt.XT_ERR_UNSUPPORTED
    assert step(xt, shapes=()) == xt.XT_OK
    n = C.c_size_t(0)
    R = (C.c_int64 * 1)(8)
    assert L.xt_muon_workspace_size(1, R, R, None) == bad and L.xt_muon_workspace_size(1, None, R, C.byref(n)) == bad
    assert L.xt_muon_workspace_size(1, R, R, C.byref(n)) == xt.XT_OK and n.value >= 8 * 64 + 8 * 64
    assert L.xt_muon_workspace_size(0, None, None, C.byref(n)) == xt.XT_OK


def test_binding_refusals(xt):
    cfg = xt.muon_config(1e-3)
    z = torch.zeros
    for args in (([z(4)], [z(4)], [z(4)]), ([z(4, 4)], [z(4, 5)], [z(4, 4)]), ([z(4, 4)], [z(4, 4)], []),
                 ([z(4, 4)], [z(4, 4)], [z(4, 4).double()]), ([z(4, 4)], [z(4, 4)], [z(4, 4)], [z(4, 5)]),
                 ([z(4, 4)], [z(4, 4).t()], [z(4, 4)])):  # the last (and all of them): not on a GPU
        with pytest.raises(ValueError):
            xt.xt_muon_step(cfg, *args)
