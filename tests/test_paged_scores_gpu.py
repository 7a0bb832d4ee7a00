"""Scores at the ends of their range: caps far above the scores, on every
kernel of the attention over a paged cache."""
from __future__ import annotations

import pytest
import torch

from gpu_util import require_cuda
from paged_util import U32, Batch, attention64, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    return require_cuda()


@pytest.fixture(scope="module")
def ws(q):
    return torch.zeros(q.PAGED_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


def shifted(t):
    """The same elements, one past a 16-byte boundary: the kernel for any
    alignment."""
    big = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    big[1:].copy_(t.reshape(-1))
    return big[1:]


def on_every_kernel(q, ws, bt, **kw):
    """(name, out, lse) of the same call on each kernel that its type has."""
    if bt.dtype != "f32":
        yield ("few rows", *run_attention(q, bt, workspace=ws, max_q_len=1, **kw))
        yield ("few rows, unsplit", *run_attention(q, bt, max_q_len=1, **kw))
        yield ("many rows", *run_attention(q, bt, workspace=ws, wide=True, **kw))
    else:
        yield ("fp32", *run_attention(q, bt, workspace=ws, **kw))
    yield ("row by row", *run_attention(q, bt, k=shifted(bt.cache(bt.k)), v=shifted(bt.cache(bt.v)), **kw))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("cap", [1e4, 1e6, 1e8, 1e30])
def test_caps_far_above_the_scores(q, ws, dtype, cap):
    """c tanh(s / c) = s - s^3 / (3 c^2) + ..: the uncapped scores to within
    2^-24 of themselves where c is 1e4 or more and |s| at most 4, so the capped
    call has to give the uncapped result.  Beside the uncapped call's roundings
    a score has at most 16 more of its own size (the quotient's, the
    polynomial's five steps', the products')."""
    bt = Batch([70, 9], [300, 40], 8, 2, 64, 16, dtype, seed=5, q_gain=0.5)
    o, l, tol, tol_l = attention64(bt)
    smax = 4.0
    big = max(float(v.abs().max()) for v in bt.vals)
    for name, out, lse in on_every_kernel(q, ws, bt, cap=cap):
        err, err_l = (out.double().cpu() - o).abs(), (lse.double().cpu() - l).abs()
        assert (err <= tol + 2 * 16 * U32 * smax * big).all(), (name, float(err.max()))
        assert (err_l <= tol_l + 16 * U32 * smax).all(), (name, float(err_l.max()))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_a_row_at_its_cap_beside_rows_far_below(q, ws, dtype):
    """One head's scores reach the cap, the other heads' of the same tokens stay
    far below it and keep their own precision."""
    cap = 1e4
    bt = Batch([64], [200], 8, 2, 64, 16, dtype, seed=6, q_gain=0.5)
    bt.q[:, 3] *= 2e4
    o, l, tol, tol_l = attention64(bt)
    small = [h for h in range(8) if h != 3]
    k = bt.keys[0][:, 0].double()
    for name, out, lse in on_every_kernel(q, ws, bt, cap=cap):
        err, err_l = (out.double().cpu() - o).abs(), (lse.double().cpu() - l).abs()
        assert (err[:, small] <= tol[:, small] + 2 * 16 * U32 * 4.0 * 5.0).all(), (name, float(err[:, small].max()))
        assert (err_l[:, small] <= tol_l[:, small] + 16 * U32 * 4.0).all(), (name, float(err_l[:, small].max()))
        for t in range(64):
            seen, x = k[:137 + t], bt.q[t, 3].double()
            s = cap * torch.tanh(x @ seen.T / 8 / cap)
            # a capped score is off by 2^-20 of the cap, a dot product by D + 4 roundings of its terms
            slack = cap * 2.0 ** -20 + 68 * U32 * float((x.abs() @ seen.abs().T).max()) / 8
            assert abs(float(lse[t, 3]) - float(torch.logsumexp(s, 0))) <= slack, (name, t)
            assert torch.isfinite(out[t, 3]).all(), (name, t)
