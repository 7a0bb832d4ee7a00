"""Paged attention on layouts a serving program has: queries inside fused rows with
a page table as wide as the sequences and far wider, and caches of up to and
beyond 32 GiB a tensor."""
from __future__ import annotations

import math

import pytest
import torch

from gpu_util import require_cuda
from paged_util import TORCH_DT, Batch, attention64, check_attention, wide_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    return require_cuda()


@pytest.fixture(scope="module")
def ws(q):
    return torch.zeros(q.PAGED_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


def attend(q, bt, ws, qd, k, v, table, strides, **kw):
    out = torch.full((bt.T, bt.Hq, bt.D), 7.0, dtype=TORCH_DT[bt.dtype], device="cuda")
    lse = torch.full((bt.T, bt.Hq), 7.0, dtype=torch.float32, device="cuda")
    q.qmv_paged_attention(qd, k, v, table.cuda(), bt.starts.cuda(), bt.lens.cuda(), out, lse, bt.T, bt.Hq, bt.Hkv, bt.D,
                          len(bt.new), bt.n_pages, bt.page, table.shape[1], 1 / math.sqrt(bt.D), bt.dtype, workspace=ws,
                          cache_strides=strides, **kw)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("new", [1, 4, 90])
@pytest.mark.parametrize("wide", [False, True])
def test_queries_inside_fused_rows(q, ws, dtype, new, wide):
    bt = Batch([new, 1], [150, 300], 8, 2, 64, 16, dtype)
    ref = attention64(bt)
    row = (bt.Hq + 2 * bt.Hkv) * bt.D
    buf = torch.full((bt.T, row), float("nan"), dtype=TORCH_DT[dtype])
    buf[:, :bt.Hq * bt.D] = bt.q.reshape(bt.T, -1)
    table = wide_table(bt) if wide else bt.table
    assert (table.shape[1] > 1000) == wide
    k, v, qd = bt.cache(bt.k), bt.cache(bt.v), buf.cuda()
    for hint in (0, 1, new, 1000):
        check_attention(bt, *attend(q, bt, ws, qd, k, v, table, bt.strides, q_strides=(row, bt.D), max_q_len=hint), ref)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("beyond", [False, True], ids=["up-to-32-GiB", "beyond"])
def test_pages_far_apart(q, ws, dtype, beyond):
    """One pool of pages whose stride is that of many layers: the last page begins
    just below 2^31 places of 16 bytes (the kernels that stream keys), or above
    (the kernel for any layout)."""
    D, page, hkv = 64, 16, 2
    es = torch.finfo(TORCH_DT[dtype]).bits // 8
    torch.cuda.empty_cache()
    for new in ([1, 1], [4, 2], [90, 33]):
        bt = Batch(new, [150, 300], 8, hkv, D, page, dtype)
        ref = attention64(bt)
        last = (1 << 35) // es + (1 << 14 if beyond else -(1 << 14))        # the last page's first element, about
        stride = last // (bt.n_pages - 1) // 64 * 64
        assert (stride * (bt.n_pages - 1) + (page - 1) * hkv * D > (1 << 35) // es) == beyond
        # the last page has to be one that holds keys
        if not (bt.table == bt.n_pages - 1).any():
            b, e = (bt.table == int(bt.table.max())).nonzero()[0].tolist()
            bt.table[b, e] = bt.n_pages - 1
            bt.store(b, bt.keys[b], bt.vals[b])
        block = page * hkv * D
        pool = torch.empty(stride * (bt.n_pages - 1) + 2 * block, dtype=TORCH_DT[dtype], device="cuda")
        for p in range(bt.n_pages):
            pool[p * stride:p * stride + block] = bt.k[p].reshape(-1).cuda()
            pool[p * stride + block:p * stride + 2 * block] = bt.v[p].reshape(-1).cuda()
        assert pool.numel() * es > 34 * 10 ** 9
        for table in (bt.table, wide_table(bt)):
            check_attention(bt, *attend(q, bt, ws, bt.q.cuda(), pool, pool[block:], table, (stride, hkv * D, D),
                                        max_q_len=max(new)), ref)
        del pool
        torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,D", [(t, d) for t in ("bf16", "f16") for d in (8, 24, 40, 72, 104, 120, 136, 200, 248)]
                         + [("f32", d) for d in (4, 12, 36, 68, 100, 132, 252)])
def test_every_padding_of_the_heads(q, ws, dtype, D):
    """Heads of whole 16 bytes that fill 64, 128 or 256 dims only in part; the
    output by odd strides inside rows whose rest stays as it is."""
    for new, kv in (([1, 2], [90, 33]), ([70, 5], [150, 64])):
        bt = Batch(new, kv, 6, 2, D, 16, dtype, seed=D)
        ref = attention64(bt)
        k, v, qd = bt.cache(bt.k), bt.cache(bt.v), bt.q.cuda()
        head, row = D + 3, 6 * (D + 3) + 5
        for table in (bt.table, wide_table(bt)):
            for w in (ws, None):
                buf = torch.full((bt.T * row + 1,), 7.0, dtype=TORCH_DT[dtype], device="cuda")
                lse = torch.full((bt.T, 6), 7.0, dtype=torch.float32, device="cuda")
                q.qmv_paged_attention(qd, k, v, table.cuda(), bt.starts.cuda(), bt.lens.cuda(), buf[1:], lse, bt.T, 6, 2, D,
                                      2, bt.n_pages, 16, table.shape[1], 1 / math.sqrt(D), dtype, cache_strides=bt.strides,
                                      out_strides=(row, head), max_q_len=max(new), workspace=w)
                torch.cuda.synchronize()
                got = buf[1:].view(bt.T, row)
                heads = got[:, :6 * head].reshape(bt.T, 6, head)
                check_attention(bt, heads[..., :D], lse, ref)
                assert (heads[..., D:] == 7).all() and (got[:, 6 * head:] == 7).all() and float(buf[0]) == 7
