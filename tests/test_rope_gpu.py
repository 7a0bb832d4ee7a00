"""The rotary rotation on the GPU against its 64-bit definition."""
from __future__ import annotations

import pytest
import torch

from gpu_util import require_cuda
from paged_util import TORCH_DT, rope64, rope_tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    return require_cuda()


def inv_freq(q, rot, **kw):
    f, m = q.qmv_rope_frequencies(rot, **kw)
    return torch.tensor(f, dtype=torch.float32), m


def check(y, x, pos, f, rot, layout, dtype, m):
    ref = rope64(x, pos, f, rot, layout, m)
    err = (y.double().cpu() - ref).abs()
    tol = rope_tol(x, ref, dtype, rot, m)
    assert (err <= tol).all(), f"worst {(err / tol.clamp_min(1e-300)).max():.3g} x the bound"
    assert torch.equal(y.cpu()[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 64, 64), (1, 40, 128, 128), (7, 3, 80, 40), (33, 5, 96, 2), (3, 2, 2, 2),
                                       (130, 1, 128, 64), (257, 11, 256, 256), (5, 7, 33, 10), (64, 1, 8, 6),
                                       (19, 70, 100, 50)])
def test_matches_definition(q, dtype, layout, T, H, D, rot):
    g = torch.Generator().manual_seed(T * 1000 + D)
    x = torch.randn(T, H, D, generator=g).to(TORCH_DT[dtype])
    pos = torch.randint(-100, 100000, (T,), generator=g, dtype=torch.int32)
    f, m = inv_freq(q, rot)
    y = torch.full((T, H, D), float("nan"), dtype=TORCH_DT[dtype], device="cuda")
    q.qmv_rope(x.cuda(), y, pos.cuda(), f.cuda(), T, H, D, rot, layout, dtype, magnitude=m)
    check(y, x, pos, f, rot, layout, dtype, m)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions_and_scaling(q, layout):
    T, H, D, rot = 48, 4, 128, 128
    g = torch.Generator().manual_seed(5)
    x = torch.randn(T, H, D, generator=g)
    pos = torch.randint(2 ** 30, 2 ** 31 - 1, (T,), generator=g, dtype=torch.int64).int()
    pos[0], pos[1] = 2 ** 31 - 1, -2 ** 31
    for kw in (dict(), dict(scaling="linear", factor=8.0), dict(scaling="base", factor=4.0),
               dict(scaling="banded", factor=16.0, original_length=4096)):
        f, m = inv_freq(q, rot, **kw)
        y = torch.empty(T, H, D, device="cuda")
        q.qmv_rope(x.cuda(), y, pos.cuda(), f.cuda(), T, H, D, rot, layout, "f32", magnitude=m)
        check(y, x, pos, f, rot, layout, "f32", m)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,shift", [("bf16", 0), ("bf16", 2), ("f16", 1), ("f32", 1)])
def test_in_place_and_strides(q, layout, dtype, shift):
    """Heads inside a wider row that starts off a 16-byte boundary."""
    T, H, D, rot, wide = 21, 6, 64, 32, 6 * 64 + 40
    g = torch.Generator().manual_seed(9)
    buf = torch.randn(T * wide + shift, generator=g).to(TORCH_DT[dtype])
    dev = buf.cuda()
    f, m = inv_freq(q, rot)
    pos = torch.arange(T, dtype=torch.int32) * 37
    view = dev[shift:]
    q.qmv_rope(view, view, pos.cuda(), f.cuda(), T, H, D, rot, layout, dtype, x_strides=(wide, D),
               y_strides=(wide, D))
    x = buf[shift:].view(T, wide)[:, :H * D].reshape(T, H, D)
    got = dev.cpu()[shift:].view(T, wide)
    check(got[:, :H * D].reshape(T, H, D), x, pos, f, rot, layout, dtype, m)
    assert torch.equal(got[:, H * D:], buf[shift:].view(T, wide)[:, H * D:])      # what lies between is untouched


def test_one_row_for_all_tokens_and_head_major(q):
    """x of token stride 0 (one row read by every token), y stored head first."""
    T, H, D = 9, 4, 64
    x = torch.randn(H, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    f, m = inv_freq(q, D)
    pos = torch.arange(T, dtype=torch.int32)
    y = torch.empty(H, T, D, dtype=torch.bfloat16, device="cuda")
    q.qmv_rope(x.cuda(), y, pos.cuda(), f.cuda(), T, H, D, D, "half", "bf16", x_strides=(0, D), y_strides=(D, T * D))
    check(y.transpose(0, 1), x[None].expand(T, H, D), pos, f, D, "half", "bf16", m)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_negative_position_is_inverse_and_gradient(q, layout):
    """<R(p) x, g> = <x, R(-p) g>: the rotation by -p is the gradient's, and
    undoes the rotation; against a difference quotient too."""
    T, H, D, rot = 6, 2, 64, 48
    gen = torch.Generator().manual_seed(4)
    x, gy, dx = (torch.randn(T, H, D, generator=gen) for _ in range(3))
    f, _ = inv_freq(q, rot)
    pos = torch.tensor([0, 1, 5, 1000, 99999, 7], dtype=torch.int32)

    def turn(v, p):
        y = torch.empty(T, H, D, device="cuda")
        q.qmv_rope(v.cuda(), y, p.cuda(), f.cuda(), T, H, D, rot, layout, "f32")
        return y.cpu()
    gx = turn(gy, -pos)
    ref = rope64(gy, -pos, f, rot, layout)
    assert ((gx.double() - ref).abs() <= rope_tol(gy, ref, "f32", rot)).all()
    # the map is linear: a step of 1 has no curvature error, only rounding
    step = (turn(x + dx, pos).double() - turn(x, pos).double()) * gy.double()
    n = T * H * D
    assert abs(step.sum() - (dx.double() * gx.double()).sum()) <= n * 16 * 2.0 ** -24 * 16
    back = turn(turn(x, pos), -pos)
    assert ((back - x).abs() <= 2 * rope_tol(x, x.double(), "f32", rot)).all()


def test_long_call_on_a_side_stream_and_captured(q):
    T, H, D = 4097, 9, 128
    x = torch.randn(T, H, D, generator=torch.Generator().manual_seed(8)).half()
    f, m = inv_freq(q, 64)
    pos = torch.arange(T, dtype=torch.int32)
    xd, pd, fd = x.cuda(), pos.cuda(), f.cuda()
    y = torch.empty_like(xd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        q.qmv_rope(xd, y, pd, fd, T, H, D, 64, "interleaved", "f16")
    for _ in range(2):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(y, x, pos, f, 64, "interleaved", "f16", m)
    y.zero_()
    torch.cuda.synchronize()
    q.qmv_rope(xd, y, pd, fd, T, H, D, 64, "interleaved", "f16", stream=s)
    s.synchronize()
    check(y, x, pos, f, 64, "interleaved", "f16", m)
