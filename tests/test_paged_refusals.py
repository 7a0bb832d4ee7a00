"""Calls of the paged-cache operators that are refused on the host (no GPU)."""
from __future__ import annotations

import pytest

from test_paged_abi import EINVAL, EUNSUP, append, attention


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
