"""Scores so large that a product's rounding is many units of log2, on every
kernel of the attention over a paged cache."""
from __future__ import annotations

import math

import pytest
import torch

from gpu_util import require_cuda
from paged_util import TORCH_DT, U32, Batch, unit
from test_paged_scores_gpu import on_every_kernel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    return require_cuda()


@pytest.fixture(scope="module")
def ws(q):
    return torch.zeros(q.PAGED_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


# (f16 queries and keys of these sizes are finite up to 2e10)
@pytest.mark.parametrize("dtype,size", [(t, s) for t in ("f16", "bf16", "f32") for s in (3e8, 1e9, 1e10, 2e10)]
                         + [("bf16", 1e11), ("f32", 1e11)])
@pytest.mark.parametrize("bias", [False, True])
def test_huge_equal_scores(q, ws, dtype, size, bias):
    """Half of the keys give the same score of about `size`, the others minus
    that: a row's output is the plain mean of the first half's values, and its
    lse the score.  (A score times log2 e / sqrt D rounds by thousands of units
    of log2 here: sum and maximum have to round it alike.)"""
    D, G = 64, 8
    bt = Batch([40, 25], [300, 129], G, 1, D, 16, dtype, q_gain=0.0)
    g = torch.Generator().manual_seed(int(size) % 1000)
    dt = TORCH_DT[dtype]
    # every head and token its own size, so that the products round both ways
    mult = (1 + torch.rand(bt.T, G, generator=g))
    bt.q[:] = 0
    dims = 60
    bt.q[..., :dims] = (math.sqrt(size / dims * 8) / 2 * mult)[..., None].to(dt)
    top = torch.tensor(2 * math.sqrt(size / dims * 8) / 2).to(dt)
    for b in range(2):
        bt.keys[b].zero_()
        bt.keys[b][0::2, :, :dims] = top
        bt.keys[b][1::2, :, :dims] = -top
        bt.store(b, bt.keys[b], bt.vals[b])
    for name, out, lse in on_every_kernel(q, ws, bt, causal=False, **(dict(slopes=[0.0] * G) if bias else {})):
        for b in range(2):
            t0, n = int(bt.starts[b]), bt.new[b]
            v = bt.vals[b][0::2, 0].double()
            want, a = v.mean(0), v.abs().mean(0)
            u = unit(dtype)
            tol = u * want.abs() + (u if dtype != "f32" else 0) * a * (1 + u) + (8 + 2 * len(v)) * U32 * a
            err = (out[t0:t0 + n].double().cpu() - want).abs()
            assert (err <= tol).all(), (name, b, float(err.max()))
            s = bt.q[t0:t0 + n, :, 0].double() * float(top) * dims / 8
            assert ((lse[t0:t0 + n].double().cpu() - s).abs() <= 80 * U32 * s + 10).all(), (name, b)
