"""Sequences that end at the last positions an int holds: a window over the end of
a cache whose table maps most of its 2^31 positions to one page."""
from __future__ import annotations

import math

import pytest
import torch

from gpu_util import require_cuda
from paged_util import TORCH_DT, Batch, attention64, check_attention, rope64, rope_tol

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1
KEEP = 300                      # positions at the end that hold keys


@pytest.fixture(scope="module")
def q():
    return require_cuda()


@pytest.fixture(scope="module")
def ws(q):
    return torch.zeros(q.PAGED_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


def far_cache(bt, length, page, shift):
    """k, v of two pages (NaN but for the last KEEP positions below `length`,
    which lie in the second), and the page table."""
    cols = -(-TOP // page)
    table = torch.zeros(1, cols, dtype=torch.int32)
    table[0, -1] = 1
    row0 = length - KEEP - (cols - 1) * page
    assert row0 >= 0
    out = []
    for t in (bt.keys[0], bt.vals[0]):
        buf = torch.full((2 * page * bt.D + shift,), float("nan"), dtype=TORCH_DT[bt.dtype], device="cuda")
        view = buf[shift:].view(2, page, 1, bt.D)
        view[1, row0:row0 + KEEP] = t.cuda()
        out.append(buf[shift:])
    return (*out, table)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("short", [0, 5, 40])
@pytest.mark.parametrize("new,page,shift", [(1, 1 << 20, 0), (90, 1 << 20, 0), (90, 786433, 0), (3, 786433, 0),
                                            (5, 1 << 20, 1)])
@pytest.mark.parametrize("kw", [dict(window=70), dict(window=33, causal=False, slopes=[0.5, 0.25, 0.125, 0.0625])],
                         ids=["causal", "not-causal"])
def test_attention_at_the_last_positions(q, ws, dtype, short, new, page, shift, kw):
    length = TOP - short
    bt = Batch([new], [KEEP], 4, 1, 64, 16, dtype, seed=short)
    ref = attention64(bt, **kw)
    k, v, table = far_cache(bt, length, page, shift)
    kw = dict(kw)
    sl = torch.tensor(kw.pop("slopes"), device="cuda") if "slopes" in kw else None
    out = torch.full((new, 4, 64), 7.0, dtype=TORCH_DT[dtype], device="cuda")
    lse = torch.full((new, 4), 7.0, device="cuda")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for w in (ws, None):
        q.qmv_paged_attention(bt.q.cuda(), k, v, table.cuda(), i32(0, new), i32(length), out, lse, new, 4, 1, 64, 1, 2,
                              page, table.shape[1], 1 / math.sqrt(64), dtype, slopes=sl, max_q_len=new, workspace=w, **kw)
        torch.cuda.synchronize()
        check_attention(bt, out, lse, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_summed_again_at_the_last_positions(q, ws, dtype):
    """An infinite value that some rows see: those rows, and the others beside
    them, are summed again."""
    new, page = 90, 1 << 20
    bt = Batch([new], [KEEP], 4, 1, 64, 16, dtype)
    bt.vals[0][KEEP - 10, 0, 3] = float("inf")
    bt.vals[0][KEEP - 200, 0, 5] = float("nan")
    kw = dict(window=150)
    ref = attention64(bt, **kw)
    k, v, table = far_cache(bt, TOP, page, 0)
    out = torch.full((new, 4, 64), 7.0, dtype=TORCH_DT[dtype], device="cuda")
    lse = torch.full((new, 4), 7.0, device="cuda")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q.qmv_paged_attention(bt.q.cuda(), k, v, table.cuda(), i32(0, new), i32(TOP), out, lse, new, 4, 1, 64, 1, 2, page,
                          table.shape[1], 1 / math.sqrt(64), dtype, max_q_len=new, workspace=ws, **kw)
    torch.cuda.synchronize()
    check_attention(bt, out, lse, ref)


def test_append_at_the_last_position(q):
    D, page, n = 64, 1 << 20, 3
    cols = -(-TOP // page)
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(n, 3 * D, generator=g).bfloat16()
    k, v = (torch.zeros(2, page, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.zeros(1, cols, dtype=torch.int32)
    table[0, -1] = 1
    f, m = q.qmv_rope_frequencies(D)
    f = torch.tensor(f)
    out = torch.empty(n, D, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q.qmv_kv_append(qkv.cuda(), k, v, table.cuda(), i32(0, n), i32(TOP), f.cuda(), out, n, 1, 1, D, D, "half", 1, 2, page,
                    cols, "bf16", magnitude=m)
    torch.cuda.synchronize()
    pos = torch.arange(TOP - n, TOP)
    rows = qkv.view(n, 3, D)
    ref = rope64(rows, pos, f, D, "half", m)
    tol = rope_tol(rows, ref, "bf16", D, m)
    at = (pos - (cols - 1) * page).tolist()
    assert ((out.cpu().double() - ref[:, 0]).abs() <= tol[:, 0]).all()
    assert ((k[1, at, 0].cpu().double() - ref[:, 1]).abs() <= tol[:, 1]).all()
    assert torch.equal(v[1, at, 0].cpu(), rows[:, 2])
    assert int((k != 0).sum()) <= n * D and not k[0].any() and not v[0].any() and not v[1, :at[0]].any() and not v[1, at[-1] + 1:].any()
