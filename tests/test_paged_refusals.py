"""Calls of the paged-cache operators that are refused on the host (no GPU)."""
from __future__ import annotations

import pytest

import weight_quantized_matrix_b200 as q
from test_paged_abi import A, EINVAL, EUNSUP, append, attention


def test_caps_whose_quotient_has_too_few_bits():
    """scale / softcap multiplies every score: a subnormal one has lost bits."""
    assert attention(T=0, scale=0.125, cap=1e36) == 0
    for scale, cap in ((0.125, 3e37), (1e-30, 1e9), (0.1, 3e38), (3e37, 3e38)):
        assert attention(T=0, scale=scale, cap=cap) == EINVAL, (scale, cap)


def test_row_counts_that_an_int_cannot_round_up():
    """Packed rows are counted in steps of up to 32 x 256."""
    most = 2 ** 31 - 1 - 33 * 256
    assert attention(T=most + 1, hq=2, hkv=2, most=1) == EUNSUP
    assert attention(T=most // 8 + 1, hq=8, most=1) == EUNSUP
    assert attention(T=2 ** 31 - 1, hq=1, hkv=1) == EUNSUP


@pytest.mark.parametrize("call", [append, attention])
def test_more_sequences_than_are_counted(call):
    assert call(T=0, n_seqs=2 ** 30) == 0
    assert call(T=0, n_seqs=2 ** 30 + 1) == EUNSUP and call(n_seqs=2 ** 31 - 1) == EUNSUP


class FakeTensor:
    """What the binding asks a tensor for."""

    def __init__(self, nbytes, whole=True, device=0):
        self.nbytes, self.whole, self.device = nbytes, whole, device

    def data_ptr(self):
        return A

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return self.whole


def test_a_workspace_tensor_that_is_too_small():
    """The kernels write all of the workspace's bytes."""
    size = q.PAGED_ATTENTION_WORKSPACE_BYTES
    assert attention(T=0, ws=FakeTensor(size)) == 0 and attention(T=0, ws=FakeTensor(size + 4096)) == 0
    for ws in (FakeTensor(size - 1), FakeTensor(0), FakeTensor(1 << 20), FakeTensor(size, whole=False)):
        assert attention(ws=ws) == EINVAL and attention(T=0, ws=ws) == EINVAL
    assert attention(T=0, ws=A) == 0                        # an address: the caller's word


def test_the_workspace_of_the_header():
    import pathlib
    import re
    text = (pathlib.Path(q.__file__).parents[1] / "include" / "qmv.h").read_text()
    m = re.search(r"#define QMV_PAGED_ATTENTION_WORKSPACE_BYTES \((\d+)u << (\d+)\)", text)
    assert int(m[1]) << int(m[2]) == q.PAGED_ATTENTION_WORKSPACE_BYTES
