"""The workspace of the sorted embedding gradient, on the host: one made for the largest batch serves every smaller one."""
import pytest


@pytest.fixture(scope="module")
def xt():
    from transformer_fwd_bwd_gb300 import build
    build.build()
    from transformer_fwd_bwd_gb300 import xt as m
    m.lib()
    return m


def size(xt, T, d):
    return xt.ws_bytes("xt_embedding_sorted_bwd_workspace_size", T, d)


# 256-column tiles: 1, 3, 4, 8, 17, 2432 and more than there are warps to fill
@pytest.mark.parametrize("d", [8, 256, 700, 768, 1024, 2048, 4129, 622592, 2000000])
def test_size_does_not_fall_as_the_batch_grows(xt, d):
    tiles = -(-d // 256)
    # all small batches, and closely around the lengths at which the pieces' length changes (4864 warps' worth of pieces)
    edges = [c * (4864 // tiles + k) for c in (8, 16, 32) for k in range(-2, 4)]
    lengths = sorted({t for t in [*range(0, 300), *range(0, 400000, 997), *(e + k for e in edges for k in range(-33, 34))]
                      if t >= 0})
    last = 0
    for T in lengths:
        n = size(xt, T, d)
        assert n >= last, (T, n, last)
        # two rows for every 8 to 32 tokens, no more than twice the piece counts' largest before the pieces grow longer
        assert -(-T // 32) * 8 * d <= n <= max(-(-T // 32), min(-(-T // 8), 2 * 4864 // tiles + 1)) * 8 * d
        last = n
