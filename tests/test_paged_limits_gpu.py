"""Paged attention at the ends of its counts: more key tiles than an int holds, and
the most query rows that a call takes."""
from __future__ import annotations

import math

import pytest
import torch

from gpu_util import require_cuda
from paged_util import unit

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    return require_cuda()


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_more_tiles_than_an_int_counts(q):
    """131088 new tokens of 16 heads on one over 2^20 cached keys: 2^31 tiles of 16
    rows and 64 keys and more.  All pages hold the same 64 keys, so a row's result
    is theirs; sequences without tokens beside it lead to these
    tiles.  A lane adds 4 weights a step and the products 16 keys a step to fp32
    sums, for 2^14 steps: 2^16 roundings of 2^-24 and 2^14 of 2^-23 (the sums of a
    product may be cut, not rounded); 68 roundings of a score's terms (about 16
    in all) are below 1e-4."""
    T, G, D, n, pages = 131088, 16, 64, 2 ** 20, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    qd = torch.randn(T, G, D, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(1, 64, 1, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    kc, vc = (t.expand(pages, -1, -1, -1).contiguous() for t in (k, v))
    seqs = 200
    table = (torch.arange(n // 64, device="cuda") % pages).int().expand(seqs, -1).contiguous()
    starts = torch.full((seqs + 1,), T, dtype=torch.int32, device="cuda")
    starts[0] = 0
    lens = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
    out = torch.full((T, G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, G), 7.0, device="cuda")
    ws = torch.zeros(q.PAGED_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    q.qmv_paged_attention(qd, kc, vc, table, starts, lens, out, lse, T, G, 1, D, seqs, pages, 64, n // 64, D ** -0.5, "bf16",
                          causal=False, max_q_len=1, workspace=ws)
    torch.cuda.synchronize()
    s = qd.double().view(-1, D) @ k.double().view(64, D).T * D ** -0.5
    p = torch.softmax(s, 1)
    o, a = p @ v.double().view(64, D), p @ v.double().view(64, D).abs()
    sums = 2.0 ** 16 * 2.0 ** -24 + 2.0 ** 14 * 2.0 ** -23
    tol = unit("bf16") * o.abs() + (unit("bf16") * 1.01 + sums + 1e-4) * a
    err = (out.double().view(-1, D) - o).abs()
    assert (err <= tol).all(), float((err / tol).max())
    want = torch.logsumexp(s, 1) + math.log(n // 64)
    assert ((lse.double().view(-1) - want).abs() <= 2.0 ** 16 * 2.0 ** -24 + 1e-4).all()


@pytest.mark.parametrize("hint", [0, 1], ids=["many-rows", "few-rows"])
def test_the_most_rows_of_a_call(q, hint):
    """2^31 - 8449 packed rows at most: one query row for all tokens (stride 0),
    every token sees the same five keys."""
    G, D = 16, 8
    T = (2 ** 31 - 8449) // G
    g = torch.Generator().manual_seed(5)
    qd = torch.randn(G, D, generator=g).bfloat16()
    k, v = (torch.randn(2, 16, 1, D, generator=g).bfloat16() for _ in range(2))
    out = torch.full((T, G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q.qmv_paged_attention(qd.cuda(), k.cuda(), v.cuda(), i32(1), i32(0, T), i32(5), out, None, T, G, 1, D, 1, 2, 16, 1,
                          D ** -0.5, "bf16", causal=False, max_q_len=hint, q_strides=(0, D))
    torch.cuda.synchronize()
    p = torch.softmax(qd.double() @ k[1, :5, 0].double().T * D ** -0.5, 1)
    o, a = p @ v[1, :5, 0].double(), p @ v[1, :5, 0].double().abs()
    assert ((out[0].double().cpu() - o).abs() <= unit("bf16") * (o.abs() + 1.01 * a) + 1e-5 * a).all()
    for part in out.split(1 << 22):
        assert torch.equal(part, out[:1].expand_as(part))
