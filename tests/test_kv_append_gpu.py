"""The append of rotated keys and of values to a paged cache, against the
64-bit definition: what is stored, where, and that nothing else is touched."""
from __future__ import annotations

import pytest
import torch

from gpu_util import require_cuda
from paged_util import TORCH_DT, Batch, rope64, rope_tol

pytestmark = pytest.mark.gpu
MARK = 3.0          # what cells that must not be written hold


@pytest.fixture(scope="module")
def q():
    return require_cuda()


def run(q, bt, rot, layout, positions=None, in_place=False, q_out=True, rotate=True, qkv_pad=0, table=None, seed=1):
    dt = TORCH_DT[bt.dtype]
    Hq, Hkv, D = bt.Hq, bt.Hkv, bt.D
    wide = (Hq + 2 * Hkv) * D + qkv_pad
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn(bt.T, wide, generator=g).to(dt)
    f, m = q.qmv_rope_frequencies(rot) if rotate else ([], 1.0)
    fd = torch.tensor(f, dtype=torch.float32)
    k = torch.full_like(bt.cache(bt.k), MARK)
    v = torch.full_like(k, MARK)
    dev = rows.cuda()
    out = dev if in_place else torch.full((bt.T, Hq, D), MARK, dtype=dt, device="cuda") if q_out else None
    q.qmv_kv_append(dev, k, v, (bt.table if table is None else table).cuda(), bt.starts.cuda(), bt.lens.cuda(),
                    fd.cuda() if rotate else None, out, bt.T, Hq, Hkv, D, rot, layout, len(bt.new), bt.n_pages,
                    bt.page, bt.max_pages, bt.dtype, magnitude=m,
                    positions=None if positions is None else positions.cuda(), qkv_stride=wide,
                    q_out_stride=wide if in_place else None, cache_strides=bt.strides)
    torch.cuda.synchronize()
    x = rows[:, :(Hq + 2 * Hkv) * D].reshape(bt.T, Hq + 2 * Hkv, D)
    if in_place:
        assert torch.equal(dev.cpu()[:, Hq * D:], rows[:, Hq * D:])
        out = dev[:, :Hq * D].reshape(bt.T, Hq, D)
    return x, out, bt.read(k), bt.read(v), fd


def check(bt, x, out, k, v, f, rot, layout, positions=None, stored=None, table=None):
    table = bt.table if table is None else table
    want_k, want_v = torch.full_like(k, MARK).double(), torch.full_like(v, MARK)
    tol = torch.zeros_like(want_k)
    place = torch.zeros(bt.T, dtype=torch.int64)
    live = torch.zeros(bt.T, dtype=torch.bool)
    for b, (n, m) in enumerate(zip(bt.new, bt.kv)):
        t0 = int(bt.starts[b])
        place[t0:t0 + n] = torch.arange(m - n, m)
        live[t0:t0 + n] = True
    at = place if positions is None else positions.long()
    turned = rope64(x, at, f, rot, layout) if f.numel() else x.double()
    t_tol = rope_tol(x, turned, bt.dtype, rot) if f.numel() else torch.zeros_like(turned)
    for b, (n, m) in enumerate(zip(bt.new, bt.kv)):
        for i in range(n):
            t, j = int(bt.starts[b]) + i, m - n + i
            if j < 0 or j // bt.page >= bt.max_pages:
                continue
            p = int(table[b, j // bt.page])
            if not 0 <= p < bt.n_pages:
                continue
            want_k[p, j % bt.page] = turned[t, bt.Hq:bt.Hq + bt.Hkv]
            tol[p, j % bt.page] = t_tol[t, bt.Hq:bt.Hq + bt.Hkv]
            want_v[p, j % bt.page] = x[t, bt.Hq + bt.Hkv:]
    assert ((k.double() - want_k).abs() <= tol).all()
    assert torch.equal(v, want_v)
    if out is not None:
        out = out.double().cpu()
        err = (out - turned[:, :bt.Hq]).abs()
        assert (err[live] <= t_tol[:, :bt.Hq][live]).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("order", ["pthd", "phtd"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("new,kv,Hq,Hkv,D,rot,page", [
    ([1], [1], 4, 1, 64, 64, 16),
    ([1] * 9, [5, 16, 17, 1, 33, 64, 2, 48, 31], 32, 8, 128, 128, 16),
    ([5, 0, 31, 2], [5, 9, 40, 300], 6, 2, 80, 40, 24),
    ([70, 3], [71, 3], 3, 3, 96, 96, 1),
    ([9], [1000], 7, 1, 33, 6, 7),
])
def test_matches_definition(q, dtype, order, layout, new, kv, Hq, Hkv, D, rot, page):
    bt = Batch(new, kv, Hq, Hkv, D, page, dtype, seed=len(kv), order=order)
    check(bt, *run(q, bt, rot, layout), rot, layout)


def test_rows_outside_the_batch_stay(q):
    bt = Batch([3, 2], [10, 2], 4, 2, 64, 16, "bf16", lead=2, tail=5)
    x, out, k, v, f = run(q, bt, 64, "half")
    check(bt, x, out, k, v, f, 64, "half")
    assert (out[:2] == MARK).all() and (out[7:] == MARK).all()


def test_in_place_padded_rows_given_positions(q):
    bt = Batch([4, 1], [20, 77], 4, 2, 64, 16, "f16")
    pos = torch.tensor([100000, 7, -3, 0, 2 ** 31 - 1], dtype=torch.int32)
    check(bt, *run(q, bt, 64, "half", positions=pos, in_place=True, qkv_pad=24), 64, "half", positions=pos)
    check(bt, *run(q, bt, 64, "half", qkv_pad=3), 64, "half")             # rows off every vector boundary


def test_without_queries_or_rotation(q):
    bt = Batch([4, 1], [20, 77], 4, 2, 64, 16, "bf16")
    check(bt, *run(q, bt, 32, "interleaved", q_out=False), 32, "interleaved")
    check(bt, *run(q, bt, 0, "half", rotate=False), 0, "half")
    none = Batch([4, 1], [20, 77], 2, 2, 64, 16, "bf16")
    none.Hq = 0
    check(none, *run(q, none, 64, "half", q_out=False), 64, "half")


def test_bad_pages_are_not_stored(q):
    """Ids outside the cache, pages past the table, more new tokens than keys."""
    bt = Batch([6, 4, 40], [30, 2, 40], 2, 2, 64, 16, "bf16")
    table = bt.table.clone()
    table[0, 1] = bt.n_pages
    table[2, 0] = -7
    bt.lens[2] = 60                                   # positions 20..59 of a table of 4 pages (64)
    bt.kv[2] = 60
    check(bt, *run(q, bt, 64, "half", table=table), 64, "half", table=table)
    bt.lens[2] = bt.kv[2] = 100                       # past the table
    check(bt, *run(q, bt, 64, "half", table=table), 64, "half", table=table)


def test_cache_beyond_32_bit_offsets(q):
    """Pages whose elements lie past 2^31."""
    D, Hkv, page = 128, 8, 64
    n_pages = 2 ** 31 // (D * Hkv * page) + 8
    k = torch.full((n_pages, page, Hkv, D), MARK, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, MARK)
    rows = torch.randn(3, (1 + 2) * Hkv * D, generator=torch.Generator().manual_seed(1)).bfloat16()
    table = torch.tensor([[n_pages - 1, n_pages - 3]], dtype=torch.int32)
    f, m = q.qmv_rope_frequencies(D)
    f = torch.tensor(f, dtype=torch.float32)
    out = torch.empty(3, Hkv, D, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q.qmv_kv_append(rows.cuda(), k, v, table.cuda(), i32(0, 3), i32(65), f.cuda(), out, 3, Hkv, Hkv, D, D, "half", 1,
                    n_pages, page, 2, "bf16")
    torch.cuda.synchronize()
    x = rows.view(3, 3 * Hkv, D)
    turned = rope64(x, torch.tensor([62, 63, 64]), f, D, "half")
    tol = rope_tol(x, turned, "bf16", D)
    for t, (p, r) in enumerate([(n_pages - 1, 62), (n_pages - 1, 63), (n_pages - 3, 0)]):
        assert ((k[p, r].cpu().double() - turned[t, Hkv:2 * Hkv]).abs() <= tol[t, Hkv:2 * Hkv]).all()
        assert torch.equal(v[p, r].cpu(), x[t, 2 * Hkv:])
    assert int((v != MARK).any(-1).any(-1).sum()) == 3
