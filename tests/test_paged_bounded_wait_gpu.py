"""The bounded waits of the attention kernel for many rows run out and report.

qmv_test_skip_last_copy leaves out the first tile of keys of block 0: the
products that need it are never issued, some warp's wait (about one second)
expires, it ORs its code into the fault word and raises the flag that ends the
other warps' waits; the block frees its tensor memory and ends, no copy is left
in flight, and the next call on the same context is right again (with a cleared
workspace)."""
from __future__ import annotations

import pytest
import torch

from gpu_util import require_cuda
from paged_util import Batch, attention64, check_attention, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    return require_cuda()


@pytest.mark.parametrize("D,page", [(128, 16), (64, 24)])
def test_wait_runs_out_and_reports(q, D, page):
    bt = Batch([300], [700], 8, 2, D, page, "bf16")
    ws = torch.zeros(q.PAGED_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    ref = attention64(bt)
    check_attention(bt, *run_attention(q, bt, workspace=ws, wide=True), ref)
    q.qmv_device_fault(clear=True)
    q.qmv_test_skip_last_copy(True)
    try:
        run_attention(q, bt, workspace=ws, wide=True)           # returns; its output is undefined
    finally:
        q.qmv_test_skip_last_copy(False)
    code = q.qmv_device_fault(clear=True)
    assert code and not code & ~(1 | 2 | 8 | 16), code
    assert q.qmv_device_fault() == 0
    ws.zero_()
    check_attention(bt, *run_attention(q, bt, workspace=ws, wide=True), ref)
    assert q.qmv_device_fault() == 0
