"""The binding's and the library's host side at the edges of their contracts, without a GPU."""
import contextlib

import pytest
import torch


@pytest.fixture(scope="module")
def xt():
    from transformer_fwd_bwd_gb300 import build
    build.build()
    from transformer_fwd_bwd_gb300 import xt as m
    m.lib()
    return m


@pytest.mark.parametrize("make", ["workspace", "scratch"])
def test_workspaces_are_made_under_the_stream_that_uses_them(xt, monkeypatch, make):
    """Allocation and fill run under the call's stream, whatever form it is given in; without one under the current."""
    inside, seen = [], []

    @contextlib.contextmanager
    def under(s):
        inside.append(s)
        yield
        inside.pop()

    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle
    for name in ("empty", "zeros"):
        plain = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, plain=plain, **kw: seen.append(tuple(inside)) or plain(*a, **kw))
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("handle", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    side = Stream(0x10)
    for s, want in ((None, ()), (side, (side,)), (0x20, (("handle", 0x20),)), (0, ("default",))):
        t = getattr(xt, make)(100, "cpu", s=s)
        assert t.numel() == 100 and seen.pop() == want and not seen


def test_every_call_gives_its_own_workspace_the_stream(xt):
    """No binding that takes ws = None and s makes the workspace without s."""
    import inspect
    import re
    made = re.findall(r"^ +ws = (\w+)\((.*)\)$", inspect.getsource(xt), re.M)
    assert len(made) >= 18
    for name, args in made:
        assert re.search(r"(\bs=s|, s)$", args), (name, args)


def test_tape_rope_axes_refuses_columns_beside_the_heads(xt):
    from transformer_fwd_bwd_gb300 import tape
    pos = torch.zeros(2, 8, dtype=torch.int32)
    for x in (torch.ones(8, 192), torch.ones(8, 64), torch.ones(8, 2, 64)):
        with pytest.raises(ValueError, match="H\\*hd"):
            tape.rope_axes(tape.leaf(x), pos, [8, 24], 2, 64)


def test_multicast_pairs_are_for_one_gpu(xt, monkeypatch):
    try:
        monkeypatch.setenv("WORLD_SIZE", "2")
        assert xt.lib().xt_gemm_set_pairing(3) == xt.XT_ERR_UNSUPPORTED
        assert b"one GPU" in xt.lib().xt_last_error()
        assert [xt.lib().xt_gemm_set_pairing(m) for m in (1, 2, 0)] == [0, 0, 0]
        monkeypatch.setenv("WORLD_SIZE", "1")
        if torch.cuda.device_count() <= 1:
            assert xt.lib().xt_gemm_set_pairing(3) == xt.XT_OK
    finally:
        xt.lib().xt_gemm_set_pairing(0)
