"""Attention over a paged cache on the GPU against its 64-bit definition."""
from __future__ import annotations

import pytest
import torch

from gpu_util import require_cuda
from paged_util import TORCH_DT, Batch, attention64, check_attention, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    return require_cuda()


@pytest.fixture(scope="module")
def ws(q):
    return torch.zeros(q.PAGED_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


def both(q, ws, bt, **kw):
    ref = attention64(bt, **{k: v for k, v in kw.items() if k not in ("q_strided", "max_q_len")})
    for w in (ws, None):
        for wide in (False, True):
            check_attention(bt, *run_attention(q, bt, workspace=w, wide=wide, **kw), ref)


# new tokens, keys, Hq, Hkv, D, page
SHAPES = [
    ([1], [1], 1, 1, 64, 16),
    ([1], [700], 32, 8, 128, 16),
    ([1] * 7, [3, 64, 65, 1, 400, 129, 16], 8, 1, 128, 16),
    ([1, 4, 2], [130, 4, 517], 16, 16, 64, 24),
    ([5, 3], [5, 260], 14, 2, 128, 1),
    ([33, 1, 70], [40, 900, 70], 12, 4, 128, 32),
    ([130], [390], 6, 2, 64, 64),
    ([300, 17], [300, 200], 4, 4, 128, 128),
    ([1, 20], [333, 150], 9, 3, 96, 8),
    ([2, 40], [50, 140], 4, 2, 256, 16),
    ([3], [90], 5, 1, 33, 7),
    ([9, 1], [70, 20], 21, 3, 80, 16),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}-{s[2]}-{s[3]}-{s[4]}-{s[5]}".replace(" ", ""))
def test_matches_definition(q, ws, dtype, shape):
    new, kv, Hq, Hkv, D, page = shape
    bt = Batch(new, kv, Hq, Hkv, D, page, dtype, seed=sum(kv), order="pthd" if Hkv % 2 else "phtd")
    both(q, ws, bt)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("new", [[1, 1, 1], [4, 1, 3], [150, 40, 1]])
@pytest.mark.parametrize("kw", [dict(window=1), dict(window=37), dict(window=300), dict(causal=False),
                                dict(causal=False, window=50), dict(cap=5.0), dict(cap=30.0, window=128),
                                dict(slopes=True), dict(slopes=True, cap=8.0, causal=False)],
                         ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_masks_and_scores(q, ws, dtype, new, kw):
    bt = Batch(new, [max(310, new[0]), max(129, new[1]), 64], 8, 2, 128, 16, dtype, seed=7)
    kw = dict(kw)
    if kw.pop("slopes", False):
        kw["slopes"] = [2.0 ** -(i + 1) for i in range(8)]
    both(q, ws, bt, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_rows_and_sequences(q, ws, dtype):
    """No keys at all, no new tokens, more new tokens than keys (their first
    ones are before position 0), rows around the batch."""
    bt = Batch([2, 0, 1, 5, 0], [0, 30, 20, 3, 0], 4, 2, 64, 16, dtype, lead=3, tail=4)
    both(q, ws, bt)
    both(q, ws, bt, causal=False)
    bt = Batch([140, 0, 3], [60, 5, 0], 4, 2, 64, 16, dtype, lead=1, tail=9)
    both(q, ws, bt)
    both(q, ws, bt, window=4)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("new", [1, 6, 200])
def test_what_a_row_does_not_see_never_reaches_it(q, ws, dtype, new):
    """NaN and infinite keys and values at later tokens, outside the window and
    in the unused part of a page (the cache's junk is NaN throughout)."""
    bt = Batch([new], [260], 4, 2, 128, 16, dtype)
    inf, nan = float("inf"), float("nan")
    if new > 2:
        # the last two new tokens: only they themselves and later ones see them
        bt.vals[0][-1, :, 5] = nan
        bt.vals[0][-2, 0, 7] = inf
        bt.keys[0][-1, 1, 3] = nan
    bt.vals[0][3, :, 2] = -inf
    bt.keys[0][4, 0, 0] = nan
    bt.store(0, bt.keys[0], bt.vals[0])
    if new <= 6:
        both(q, ws, bt, window=100)
    else:
        both(q, ws, bt, window=40)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
def test_a_value_that_all_rows_see(q, ws, dtype, D):
    """An infinite and a NaN value far back in a long context: every row of a
    chunk is summed again exactly, in all its parts."""
    bt = Batch([90, 40], [9000, 700], 4, 2, D, 16, dtype)
    bt.vals[0][17, 0, 3], bt.vals[0][8000, 1, 5], bt.vals[1][650, :, 7] = float("inf"), float("nan"), -float("inf")
    for b in range(2):
        bt.store(b, bt.keys[b], bt.vals[b])
    both(q, ws, bt)
    both(q, ws, bt, window=500, cap=20.0)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_lowest_and_infinite_scores(q, ws, dtype):
    """Scores of the type's lowest value, all scores -infinity (zeros), one
    +infinity among finite ones (NaN, as in the definition)."""
    big = torch.finfo(TORCH_DT[dtype]).max
    bt = Batch([2], [50], 2, 1, 64, 16, dtype, q_gain=0.0)
    bt.q[:, 0, 0], bt.q[:, 1, 0] = 1.0, -1.0
    bt.keys[0].zero_()
    bt.keys[0][:, 0, 0] = big
    bt.store(0, bt.keys[0], bt.vals[0])
    both(q, ws, bt)
    bt.keys[0][:, 0, 0] = float("inf")
    bt.store(0, bt.keys[0], bt.vals[0])
    out, lse = run_attention(q, bt, workspace=ws)
    assert torch.isnan(out[:, 0]).all() and torch.isnan(lse[:, 0]).all()
    assert (out[:, 1] == 0).all() and (lse[:, 1] == -float("inf")).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,wide", [(1, False), (3, False), (150, False), (150, True)])
def test_bad_pages_make_their_rows_nan(q, ws, dtype, new, wide):
    bt = Batch([new, new], [200, 200], 4, 2, 128, 16, dtype)
    ref = attention64(bt)
    bt.table[0, 6] = bt.n_pages                                   # positions 96..111 of the first sequence
    out, lse = run_attention(q, bt, workspace=ws, wide=wide)
    sees = torch.arange(200 - new, 200) >= 96
    assert torch.isnan(out[:new].cpu()[sees]).all() and torch.isnan(lse[:new].cpu()[sees]).all()
    o, l, tol, tl = ref
    keep = torch.cat([~sees, torch.ones(new, dtype=torch.bool)])
    assert ((out.cpu().double() - o).abs() <= tol)[keep].all()
    # a window that ends behind the bad page does not see it
    kw = dict(window=60)
    ref = attention64(bt, **kw)
    out, lse = run_attention(q, bt, workspace=ws, wide=wide, **kw)
    keep = torch.cat([(torch.arange(200 - new, 200) < 96) | (torch.arange(200 - new, 200) - 60 >= 111),
                      torch.ones(new, dtype=torch.bool)])
    assert ((out.cpu().double() - ref[0]).abs() <= ref[2])[keep].all()
    # keys past the table
    bt.lens[1] = bt.max_pages * bt.page + 5
    out, _ = run_attention(q, bt, workspace=ws)
    assert torch.isnan(out[new + new - 1].float()).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("new,wide", [(1, False), (90, False), (90, True)])
def test_strides_alignment_and_hints(q, ws, dtype, new, wide):
    """Queries inside fused rows; a wrong or absent max_q_len; no lse; a cache
    that starts off a 16-byte boundary."""
    bt = Batch([new, 1], [150, 300], 8, 2, 64, 16, dtype)
    ref = attention64(bt)
    for hint in (0, 1, 1000):
        check_attention(bt, *run_attention(q, bt, workspace=ws, max_q_len=hint, q_strided=True, wide=wide), ref)
    check_attention(bt, *run_attention(q, bt, workspace=ws, lse=False, wide=wide), ref)

    def shifted(t):
        b = bt.cache(t)
        big = torch.empty(b.numel() + 1, dtype=b.dtype, device="cuda")
        big[1:].copy_(b.reshape(-1))
        return big[1:]
    check_attention(bt, *run_attention(q, bt, workspace=ws, k=shifted(bt.k), v=shifted(bt.v), wide=wide), ref)


def test_long_context_split_and_repeatable(q, ws):
    """One token over many keys: the split over blocks, the same twice, and the
    workspace left ready for a call of another size."""
    for dtype, new in (("bf16", [1, 2]), ("f32", [1, 2]), ("bf16", [70, 20]), ("f16", [300, 1])):
        bt = Batch(new, [9000, 3333], 8, 2, 128, 64, dtype, seed=3)
        ref = attention64(bt)
        a = run_attention(q, bt, workspace=ws)
        check_attention(bt, *a, ref)
        small = Batch([1], [33], 2, 1, 64, 16, dtype)
        check_attention(small, *run_attention(q, small, workspace=ws), attention64(small))
        b = run_attention(q, bt, workspace=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_many_sequences(q, ws):
    """More sequences than a block has threads."""
    n = 700
    g = torch.Generator().manual_seed(2)
    kv = torch.randint(1, 40, (n,), generator=g).tolist()
    bt = Batch([1] * n, kv, 4, 1, 64, 16, "bf16")
    both(q, ws, bt)
    new = [min(k, 1 + i % 3) if i % 5 else 0 for i, k in enumerate(kv)]
    bt = Batch(new, kv, 16, 1, 64, 16, "bf16")
    both(q, ws, bt, max_q_len=100)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("new", [[1100, 3], [5, 0, 1030, 64, 90] + [37, 1] * 8, [1, 5, 2, 40] * 45],
                         ids=["one-long", "20-ragged", "180-ragged"])
def test_many_units_a_sequence(q, ws, dtype, new):
    """Sequences of more row tiles than a warp has lanes, in batches that give a
    sequence 32, a few or one of a block's threads to count them."""
    kv = [n + 17 * (i % 7) for i, n in enumerate(new)]
    bt = Batch(new, kv, 8, 1, 64, 16, dtype, seed=len(new))
    both(q, ws, bt)
    both(q, ws, bt, window=45)
    ref = attention64(bt)
    for hint in (1, 4000):                      # both kernels of the 16-bit types
        check_attention(bt, *run_attention(q, bt, workspace=ws, max_q_len=hint), ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed_with_new_lengths(q, ws, dtype):
    """A captured call reads the lengths on the device at each replay."""
    bt = Batch([1, 1], [100, 260], 8, 2, 128, 16, dtype)
    k, v = bt.cache(bt.k), bt.cache(bt.v)
    table, starts, lens, qd = bt.table.cuda(), bt.starts.cuda(), bt.lens.cuda(), bt.q.cuda()
    out = torch.empty_like(qd)
    lse = torch.empty(2, 8, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        q.qmv_paged_attention(qd, k, v, table, starts, lens, out, lse, 2, 8, 2, 128, 2, bt.n_pages, 16, bt.max_pages,
                              128 ** -0.5, dtype, max_q_len=1, cache_strides=bt.strides, workspace=ws)
    for cut in (0, 70, 99):
        lens.copy_(bt.lens - cut)
        g.replay()
        torch.cuda.synchronize()
        part = Batch([1, 1], [100 - cut, 260 - cut], 8, 2, 128, 16, dtype)
        part.q = bt.q
        part.keys, part.vals = ([t[:n] for t, n in zip(s, part.kv)] for s in (bt.keys, bt.vals))
        check_attention(part, out, lse, attention64(part))


def test_first_call_of_a_process_may_be_captured():
    """Nothing has to run before a capture."""
    code = '''
import torch, weight_quantized_matrix_b200 as q
i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
for T, wide in ((1, 13), (200, 40000)):
    qkv = torch.randn(T, 8 * 64, device="cuda").bfloat16()
    k, v = (torch.zeros(20, 16, 2, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = torch.zeros(1, wide, dtype=torch.int32, device="cuda")
    table[0, :13] = torch.arange(13, device="cuda")
    starts, lens, f = i32(0, T), i32(T), torch.ones(32, device="cuda")
    qr, out = (torch.empty(T, 4, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    ws = torch.zeros(q.PAGED_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qmv_kv_append(qkv, k, v, table, starts, lens, f, qr, T, 4, 2, 64, 64, "half", 1, 20, 16, wide, "bf16")
        q.qmv_paged_attention(qr, k, v, table, starts, lens, out, None, T, 4, 2, 64, 1, 20, 16, wide, 0.125, "bf16", workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all() and (out != 0).any()
    if T == 1:
        assert torch.equal(out[0].view(2, 2, 64), qkv[0, 6 * 64:].view(2, 1, 64).expand(2, 2, 64))   # one key: its value
print("captured")
'''
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_streams_with_their_own_workspaces(q):
    bts = [Batch([1, 3], [2000 + 500 * i, 90], 8, 2, 128, 16, "bf16", seed=i) for i in range(2)]
    refs = [attention64(bt) for bt in bts]
    for _ in range(3):
        streams = [torch.cuda.Stream() for _ in bts]
        w = [torch.zeros(q.PAGED_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda") for _ in bts]
        torch.cuda.synchronize()
        got = [run_attention(q, bt, workspace=x, stream=s) for bt, x, s in zip(bts, w, streams)]
        for bt, o, ref in zip(bts, got, refs):
            check_attention(bt, *o, ref)
