"""Softmax weights far below the largest, on every kernel of the attention over a
paged cache."""
from __future__ import annotations

import math

import pytest
import torch

from gpu_util import require_cuda
from paged_util import U32, Batch, attention64
from test_paged_scores_gpu import on_every_kernel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    return require_cuda()


@pytest.fixture(scope="module")
def ws(q):
    return torch.zeros(q.PAGED_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("low", [15, 24, 27])
@pytest.mark.parametrize("kw", [dict(), dict(cap=1e4)], ids=["plain", "capped"])
def test_one_large_weight_and_a_long_flat_tail(q, ws, dtype, low, kw):
    """The first 128 keys, whose values are 0, take almost all of the weight; thousands of
    keys at 2^-low of it make the whole output, and f16 holds nothing below 2^-24
    by itself.  Its weights are held to half a unit of themselves and 2^-32 of
    the row's largest."""
    n = 4000
    bt = Batch([3, 80], [n, n], 4, 2, 64, 16, dtype, q_gain=0.0)
    bt.q[..., 0] = 8.0
    # scores q k / 8 in units of 1; the tail at -low log 2, in steps the type holds
    for b in range(2):
        bt.keys[b].zero_()
        bt.keys[b][128:, :, 0] = -round(low * math.log(2) * 16) / 16
        bt.vals[b].abs_().mul_(500).add_(500)
        bt.vals[b][:128] = 0
        bt.store(b, bt.keys[b], bt.vals[b])
    o, l, tol, tol_l = attention64(bt)
    if dtype == "f16":
        every = torch.cat([v.double().sum(0).mul(2.0 ** -32).repeat_interleave(2, 0)[None].expand(m, -1, -1)
                           for v, m in zip(bt.vals, bt.new)])
        tol = tol + every / torch.exp(l)[..., None]            # the largest score is 0
    tol = tol + 2 * 16 * U32 * 20 * o.abs()
    assert (tol <= 0.06 * o.abs()).all()
    for name, out, lse in on_every_kernel(q, ws, bt, **kw):
        assert ((out.double().cpu() - o).abs() <= tol).all(), (name, float((out.double().cpu() / o - 1).abs().max()))
        assert ((lse.double().cpu() - l).abs() <= tol_l + 16 * U32 * 20).all(), name
