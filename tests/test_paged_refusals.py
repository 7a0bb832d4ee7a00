"""Calls of the paged-cache operators that are refused on the host (no GPU)."""
from __future__ import annotations

from test_paged_abi import EINVAL, attention


def test_caps_whose_quotient_has_too_few_bits():
    """scale / softcap multiplies every score: a subnormal one has lost bits."""
    assert attention(T=0, scale=0.125, cap=1e36) == 0
    for scale, cap in ((0.125, 3e37), (1e-30, 1e9), (0.1, 3e38), (3e37, 3e38)):
        assert attention(T=0, scale=scale, cap=cap) == EINVAL, (scale, cap)
