"""GPU parity of the rotary positions over several axes (xt_rope_axes_fwd / _bwd) against the rotation in
64 bits.

Tolerance, per element y = u cos θ ∓ w sin θ, against |u| + |w|: the angle as a float32 half-turn is off by
at most 2⁻²⁴ (π·2⁻²⁴ rad), cos and sin by at most 2 ulp (2⁻²²), two products and a sum round to float32
(3·2⁻²⁴): 7.5e-7 in all; for bf16 half a step of the result (2⁻⁸ relative) on top."""
import numpy as np
import pytest
import torch

from tests.gpu_util import empty, host

pytestmark = pytest.mark.gpu

xt = pytest.importorskip("transformer_fwd_bwd_gb300.xt")

TD = {"f32": torch.float32, "bf16": torch.bfloat16}


def angles(pos, sections, hd, base, per_axis):
    """[T, hd/2] in float64."""
    out, i = [], 0
    for a, n in enumerate(sections):
        for k in range(n):
            f = base ** (-k / n if per_axis else -2.0 * i / hd)
            out.append(pos[a].astype(np.float64) * f)
            i += 1
    return np.stack(out, 1)


def rotate(x, th, H, hd, sign):
    T, h = x.shape[0], hd // 2
    v = x.reshape(T, H, hd)
    a, b = v[..., :h], v[..., h:]
    c, s = np.cos(th)[:, None], sign * np.sin(th)[:, None]
    y = np.concatenate([a * c - b * s, b * c + a * s], -1)
    mag = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
    return y.reshape(T, H * hd), mag.reshape(T, H * hd)


def compare(got, want, mag, dtype, extra=0.0):
    tol = (7.5e-7 + extra) * mag + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0.0)
    assert np.all(np.abs(host(got) - want) <= tol), float(np.max(np.abs(host(got) - want) / np.maximum(tol, 1e-30)))


def data(T, cols, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, cols, generator=g, device="cuda").to(TD[dtype])


CASES = [  # T, H, hd, sections, per_axis, dtype
    (1, 1, 2, [1], 0, "f32"),
    (5, 3, 6, [1, 2], 1, "bf16"),
    (33, 24, 64, [8, 12, 12], 0, "bf16"),
    (130, 5, 80, [10, 0, 14, 16], 1, "f32"),
    (257, 2, 128, [16, 24, 24], 0, "f32"),
    (1000, 9, 96, [48], 0, "bf16"),
    (7, 1, 256, [64, 64], 1, "bf16"),
]


@pytest.mark.parametrize("T,H,hd,sections,per_axis,dtype", CASES)
def test_forward_and_gradient(T, H, hd, sections, per_axis, dtype):
    rng = np.random.default_rng(T + hd)
    pos = rng.integers(-1000000, 1000000, size=(len(sections), T)).astype(np.int32)
    P = torch.tensor(pos, device="cuda")
    th = angles(pos, sections, hd, 10000.0, per_axis)
    x, d = data(T, H * hd, dtype, 1), data(T, H * hd, dtype, 2)
    y, dx = empty((T, H * hd), dtype), empty((T, H * hd), dtype)
    xt.xt_rope_axes_fwd(x, y, P, sections, H, hd, 10000.0, per_axis)
    xt.xt_rope_axes_bwd(d, dx, P, sections, H, hd, 10000.0, per_axis)
    # a float64 angle of up to 1e6 rad is itself off by 1e6·2⁻⁵³ in the reference and the frequency
    compare(y, *rotate(host(x), th, H, hd, 1.0), dtype, extra=1e-9)
    compare(dx, *rotate(host(d), th, H, hd, -1.0), dtype, extra=1e-9)
    # the gradient against differences: y is linear in x, so dx·v = d·(rotation of v)
    v = data(T, H * hd, dtype, 3)
    rv = rotate(host(v), th, H, hd, 1.0)[0]
    want = rotate(host(d), th, H, hd, -1.0)[0]
    assert abs(np.sum(want * host(v)) - np.sum(host(d) * rv)) <= 1e-9 * np.sum(np.abs(want * host(v)))
    # accumulation: two pushes are twice the gradient to the storage's rounding
    acc = empty((T, H * hd), dtype, fill=0.0)
    acc.copy_(dx)
    xt.xt_rope_axes_bwd(d, acc, P, sections, H, hd, 10000.0, per_axis, acc=1)
    tol = 4 * (7.5e-7 + 1e-9) * rotate(host(d), th, H, hd, -1.0)[1] + (3 * 2.0 ** -8 * np.abs(2 * want) if dtype == "bf16" else 0.0)
    assert np.all(np.abs(host(acc) - 2 * want) <= tol)


def test_one_axis_equals_rope():
    """Positions 0 .. S−1 on one axis are xt_rope_fwd's."""
    B, S, H, hd = 2, 77, 3, 64
    x = data(B * S, H * hd, "f32", 4)
    table = torch.empty(S * hd, device="cuda")
    xt.xt_rope_table(table, S, hd, 10000.0)
    a, b = empty((B * S, H * hd)), empty((B * S, H * hd))
    xt.xt_rope_fwd(x, a, table, B, S, H, hd, H * hd)
    pos = torch.arange(S, dtype=torch.int32, device="cuda").repeat(B)[None]
    xt.xt_rope_axes_fwd(x, b, pos.contiguous(), [hd // 2], H, hd)
    mag = rotate(host(x), np.zeros((B * S, hd // 2)), H, hd, 1.0)[1]
    assert np.all(np.abs(host(a) - host(b)) <= 1.1e-6 * mag)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_columns_in_place_and_misaligned(dtype):
    """Query and key heads rotated in place in a packed [q | k | v] buffer: the value columns stay as they
    were; a start that is not 16-byte aligned takes the element path with the same results."""
    T, H, hd = 50, 4, 64
    rng = np.random.default_rng(5)
    pos = torch.tensor(rng.integers(0, 5000, size=(3, T)).astype(np.int32), device="cuda")
    buf = empty((T, 3 * H * hd), dtype)
    src = data(T, 3 * H * hd, dtype, 6)
    buf.copy_(src)
    xt.xt_rope_axes_fwd(buf, buf, pos, [8, 12, 12], 2 * H, hd)
    out = empty((T, 2 * H * hd), dtype)
    xt.xt_rope_axes_fwd(src[:, :2 * H * hd], out, pos, [8, 12, 12], 2 * H, hd)
    assert torch.equal(buf[:, :2 * H * hd], out) and torch.equal(buf[:, 2 * H * hd:], src[:, 2 * H * hd:])
    wide = torch.zeros(T, 2 * H * hd + 9, dtype=TD[dtype], device="cuda")
    wide[:, 1:2 * H * hd + 1] = src[:, :2 * H * hd]
    xt.xt_rope_axes_fwd(wide[:, 1:2 * H * hd + 1], wide[:, 1:2 * H * hd + 1], pos, [8, 12, 12], 2 * H, hd)
    assert torch.equal(wide[:, 1:2 * H * hd + 1], out)
    assert not bool(wide[:, 0].any()) and not bool(wide[:, 2 * H * hd + 1:].any())


def test_extreme_positions():
    """f = 1 (one pair): the angle is the position itself; float64 reduces it correctly.  1/2π as a double
    leaves 2⁻⁵⁶ turns per position: 2π·2⁻²⁵ rad at 2³¹."""
    pos = np.array([[0, 1, -1, 2**31 - 1, -2**31, 1234567890, -987654321]], dtype=np.int32)
    x = data(7, 2, "f32", 7)
    y = empty((7, 2))
    xt.xt_rope_axes_fwd(x, y, torch.tensor(pos, device="cuda"), [1], 1, 2)
    compare(y, *rotate(host(x), pos.T.astype(np.float64), 1, 2, 1.0), "f32", extra=2 * np.pi * 2.0 ** -25)


def test_other_stream_and_capture():
    T, H, hd = 300, 6, 64
    pos = torch.arange(3 * T, dtype=torch.int32, device="cuda").view(3, T)
    x = data(T, H * hd, "bf16", 8)
    want = empty((T, H * hd), "bf16")
    xt.xt_rope_axes_fwd(x, want, pos, [8, 12, 12], H, hd)
    y = empty((T, H * hd), "bf16", fill=0.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        xt.xt_rope_axes_fwd(x, y, pos, [8, 12, 12], H, hd, s=s)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    y.zero_()
    with torch.cuda.graph(g):
        xt.xt_rope_axes_fwd(x, y, pos, [8, 12, 12], H, hd)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
