"""Arguments that the gated feed-forward block refuses, on the host: every refusal comes before anything touches a
device."""
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


def fwd(xt, x=16, wu=16, wd=16, gu=16, h=16, y=16, T=64, d=64, F=128, act=0, dt=1, ws=None, wb=0):
    return xt.lib().xt_gated_mlp_fwd(x, wu, wd, gu, h, y, T, d, F, act, dt, ws, wb, None)


def bwd(xt, x=16, wu=16, wd=16, gu=16, h=16, y=16, T=64, d=64, F=128, act=0, dt=1, ws=None, wb=0, dgu=16, dx=16, dwu=16,
        dwd=16, dg=0, ax=0, aw=0):
    return xt.lib().xt_gated_mlp_bwd(x, wu, wd, gu, h, y, dgu, dx, dwu, dwd, T, d, F, act, dt, dg, ax, aw, ws, wb, None)


@pytest.mark.parametrize("f", [fwd, bwd])
def test_refusals(xt, f):
    bad, ali = xt.XT_ERR_INVALID_ARG, xt.XT_ERR_ALIGNMENT
    assert f(xt, T=-1) == bad and f(xt, d=0) == bad and f(xt, F=0) == bad and f(xt, T=1 << 30) == bad
    assert f(xt, act=2) == bad and f(xt, act=-1) == bad
    assert f(xt, d=60) == ali and f(xt, F=132) == ali
    assert f(xt, dt=0) == xt.XT_ERR_UNSUPPORTED
    for name in ("x", "wu", "wd", "h"):
        assert f(xt, **{name: None}) == bad and f(xt, **{name: 24}) == ali
    assert f(xt, y=24) == ali and f(xt, gu=24) == ali and f(xt, ws=24, wb=1 << 20) == ali


def test_more_refusals(xt):
    bad, ali = xt.XT_ERR_INVALID_ARG, xt.XT_ERR_ALIGNMENT
    assert bwd(xt, y=None) == bad and bwd(xt, gu=None) == bad and bwd(xt, dgu=None) == bad and bwd(xt, dgu=8) == ali
    assert bwd(xt, dg=2) == bad and bwd(xt, ax=2) == bad and bwd(xt, aw=-1) == bad
    assert bwd(xt, dx=8) == ali and bwd(xt, dwu=8) == ali and bwd(xt, dwd=8) == ali
    assert fwd(xt, T=0, x=None, wu=None, h=None) == xt.XT_OK
    n = C.c_size_t(0)
    L = xt.lib()
    assert L.xt_gated_mlp_workspace_size(64, 64, 128, None) == bad
    assert L.xt_gated_mlp_workspace_size(64, 60, 128, C.byref(n)) == ali
    assert L.xt_gated_mlp_workspace_size(64, 64, 128, C.byref(n)) == xt.XT_OK and n.value >= 4096
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    good = dict(x=z(4, 16), w_up=z(16, 48), w_down=z(24, 16), gu=z(4, 48), h=z(4, 24), y=z(4, 16))
    for change in (dict(x=z(4, 8)), dict(w_up=z(16, 47)), dict(w_down=z(24, 8)), dict(gu=z(4, 24)), dict(h=z(5, 24)),
                   dict(y=z(4, 24)), dict(h=z(4, 24).float()), dict(y=None), {}):  # the last: not on a GPU
        with pytest.raises(ValueError):
            xt.xt_gated_mlp_fwd(**{**good, **change})
    more = dict(good, dy=z(4, 16), dgu=z(4, 48), dx=z(4, 16), dw_up=z(16, 48), dw_down=z(24, 16))
    del more["y"]
    for change in (dict(dw_up=z(16, 48).float()), dict(dx=z(4, 24)), dict(dgu=z(4, 24)), dict(dy=z(4, 16).float())):
        with pytest.raises(ValueError):
            xt.xt_gated_mlp_bwd(**{**more, **change})
