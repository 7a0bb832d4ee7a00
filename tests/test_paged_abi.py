"""Rotation, append and paged attention without a GPU: refusals happen on the
host before any launch, and the frequencies follow their formulas."""
from __future__ import annotations

import ctypes
import math

import pytest

import weight_quantized_matrix_b200 as q

EINVAL, EUNSUP, EALIGN = -1, -2, -3
A, B = 1 << 20, 1 << 40          # aligned fake addresses far apart: refused calls never touch them


def status(fn, *a, **kw):
    try:
        fn(*a, **kw)
    except q.QmvError as e:
        return e.status
    return 0


def rope(**kw):
    a = dict(x=A, y=B, pos=A, f=A, T=2, H=4, D=64, rot=64, layout="half", dtype="bf16", xs=None, ys=None)
    a.update(kw)
    return status(q.qmv_rope, a["x"], a["y"], a["pos"], a["f"], a["T"], a["H"], a["D"], a["rot"], a["layout"],
                  a["dtype"], x_strides=a["xs"], y_strides=a["ys"], stream=0)


def test_rope_refusals():
    assert rope(T=0) == 0 and rope(H=0) == 0 and rope(T=0, x=None, y=None, pos=None, f=None) == 0
    assert rope(dtype=3) == EUNSUP and rope(layout=2) == EUNSUP and rope(D=257, rot=64) == EUNSUP
    for bad in (dict(T=-1), dict(H=-1), dict(D=0), dict(rot=0), dict(rot=3), dict(rot=66), dict(rot=-2)):
        assert rope(**bad) == EINVAL, bad
    for name in ("x", "y", "pos", "f"):
        assert rope(**{name: None}) == EINVAL
    for name, off in (("x", 1), ("y", 1), ("pos", 2), ("f", 2)):
        assert rope(**{name: A + off if name != "y" else B + off}) == EALIGN
    assert rope(xs=(-1, 64)) == EINVAL and rope(xs=(256, -64)) == EINVAL
    for ys in ((64, 64), (255, 64), (256, 63), (0, 64), (32, 128), (-256, 64)):
        assert rope(ys=ys) == EINVAL, ys                    # rows of y that share elements
    assert rope(y=A + 64) == EINVAL                          # y meets x
    assert rope(y=A, ys=(512, 64)) == EINVAL


CACHE = dict(k=A, v=A, table=A, starts=A, lens=A, hkv=2, D=64, n_seqs=2, n_pages=9, page=16, max_pages=4, dtype="bf16",
             cs=None)


def append(**kw):
    a = dict(CACHE, qkv=A, f=A, out=B, T=3, hq=4, rot=64, layout="half", pos=None, qs=None, os=None)
    a.update(kw)
    return status(q.qmv_kv_append, a["qkv"], a["k"], a["v"], a["table"], a["starts"], a["lens"], a["f"], a["out"],
                  a["T"], a["hq"], a["hkv"], a["D"], a["rot"], a["layout"], a["n_seqs"], a["n_pages"], a["page"],
                  a["max_pages"], a["dtype"], positions=a["pos"], qkv_stride=a["qs"], q_out_stride=a["os"],
                  cache_strides=a["cs"], stream=0)


def attention(**kw):
    a = dict(CACHE, q=A, out=B, lse=A, T=3, hq=4, scale=0.1, causal=True, window=0, cap=0.0, slopes=None, most=0,
             qs=None, os=None, ws=None)
    a.update(kw)
    return status(q.qmv_paged_attention, a["q"], a["k"], a["v"], a["table"], a["starts"], a["lens"], a["out"], a["lse"],
                  a["T"], a["hq"], a["hkv"], a["D"], a["n_seqs"], a["n_pages"], a["page"], a["max_pages"], a["scale"],
                  a["dtype"], causal=a["causal"], window=a["window"], softcap=a["cap"], slopes=a["slopes"],
                  max_q_len=a["most"], cache_strides=a["cs"], q_strides=a["qs"], out_strides=a["os"],
                  workspace=a["ws"], stream=0)


@pytest.mark.parametrize("call", [append, attention])
def test_cache_refusals(call):
    assert call(T=0) == 0 and call(n_seqs=0) == 0
    assert call(T=0, k=None, table=None) == 0
    assert call(dtype=7) == EUNSUP and call(D=260, rot=64) == EUNSUP
    for bad in (dict(T=-1), dict(n_seqs=-1), dict(n_pages=0), dict(page=0), dict(hkv=0), dict(D=0), dict(max_pages=0)):
        assert call(**bad) == EINVAL, bad
    for name in ("k", "v", "table", "starts", "lens"):
        assert call(**{name: None}) == EINVAL, name
        assert call(**{name: A + 1}) == EALIGN, name
    # cache rows that share elements
    for cs in ((0, 128, 64), (2048, 64, 64), (2048, 127, 64), (1024, 128, 64), (-2048, 128, 64), (2048, 128, 32)):
        assert call(cs=cs) == EINVAL, cs


def test_append_refusals():
    assert append(qkv=None) == EINVAL and append(qkv=A + 1) == EALIGN and append(out=B + 1) == EALIGN
    assert append(f=A + 2) == EALIGN and append(pos=A + 2) == EALIGN
    for bad in (dict(hq=-1), dict(rot=0), dict(rot=7), dict(rot=66), dict(qs=8 * 64 - 1), dict(os=255),
                dict(hq=0), dict(out=A + 128), dict(out=A, os=1024)):
        assert append(**bad) == EINVAL, bad
    assert append(layout=9) == EUNSUP


def test_attention_refusals():
    assert attention(q=None) == EINVAL and attention(out=None) == EINVAL
    for name in ("q", "lse", "slopes"):
        assert attention(**{name: A + 1}) == EALIGN
    assert attention(ws=A + 8) == EALIGN and attention(out=B + 1) == EALIGN
    for bad in (dict(hq=0), dict(hq=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")),
                dict(scale=3e38), dict(scale=1.0, cap=1e-39), dict(window=-1), dict(most=-1), dict(qs=(-1, 64)), dict(os=(255, 64)), dict(os=(256, 0))):
        assert attention(**bad) == EINVAL, bad


def test_too_many_rows():
    assert attention(T=2 ** 28, hq=8, most=1) == EUNSUP


def test_host_tensors_are_refused():
    import torch
    t = torch.zeros(4, 4, 64)
    assert rope(x=t) == EINVAL and rope(y=t) == EINVAL
    assert append(qkv=t) == EINVAL and append(k=t) == EINVAL
    assert attention(q=t) == EINVAL and attention(out=t) == EINVAL


def test_a_size_beyond_int_is_not_narrowed():
    with pytest.raises(OverflowError):
        rope(T=2 ** 32 + 1)
    with pytest.raises(OverflowError):
        attention(T=2 ** 32 + 1)


def test_null_cache():
    lib = q.lib()
    lib.qmv_paged_attention.argtypes = [ctypes.c_void_p] * 4 + [ctypes.c_int] * 2 + [ctypes.c_float] + [
        ctypes.c_int] * 2 + [ctypes.c_float, ctypes.c_void_p] + [ctypes.c_longlong] * 4 + [ctypes.c_int] + [
        ctypes.c_void_p] * 2
    assert lib.qmv_paged_attention(A, None, B, None, 1, 1, 1.0, 1, 0, 0.0, None, 64, 64, 64, 64, 0, None, None) == EINVAL


# ------------------------------------------------------------- frequencies ---
def test_plain_and_linear_frequencies():
    f, m = q.qmv_rope_frequencies(128, 500000.0)
    assert m == 1.0 and len(f) == 64
    for i, v in enumerate(f):
        want = 500000.0 ** (-2 * i / 128)
        assert abs(v - want) <= 2.0 ** -24 * want * (1 + 1e-6)
    g, m = q.qmv_rope_frequencies(128, 500000.0, "linear", 8.0)
    assert m == 1.0 and all(a == b * 8 for a, b in zip(f, g))       # a power of two: exact


def test_base_scaling_stretches_the_slowest_pair_only():
    f, _ = q.qmv_rope_frequencies(64)
    g, m = q.qmv_rope_frequencies(64, scaling="base", factor=4.0)
    assert m == 1.0 and g[0] == f[0] == 1.0
    assert abs(f[-1] / g[-1] - 4.0) < 1e-5
    assert all(a >= b for a, b in zip(f, g))


def test_banded_scaling():
    n, factor = 4096, 16.0
    f, _ = q.qmv_rope_frequencies(128)
    g, m = q.qmv_rope_frequencies(128, scaling="banded", factor=factor, original_length=n)
    assert abs(m - (0.1 * math.log(factor) + 1)) < 1e-6
    kept = stretched = 0
    for a, b in zip(f, g):
        turns = a * n / (2 * math.pi)
        ratio = a / b
        assert 1 - 1e-6 <= ratio <= factor * (1 + 1e-6)
        if turns > 32 * 1.2:
            assert abs(ratio - 1) < 1e-6
            kept += 1
        if turns < 1 / 1.2:
            assert abs(ratio - factor) < 1e-4
            stretched += 1
    assert kept > 5 and stretched > 5
    ratios = [a / b for a, b in zip(f, g)]
    assert all(x <= y * (1 + 1e-6) for x, y in zip(ratios, ratios[1:]))


def test_frequency_refusals():
    fn = q.qmv_rope_frequencies
    assert status(fn, 128, scaling=4) == EUNSUP and status(fn, 128, scaling=-1) == EUNSUP
    for bad in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=-2), dict(base=1.0), dict(base=float("nan")),
                dict(base=float("inf")), dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("nan")),
                dict(rot_dim=2, scaling="base", factor=2.0), dict(scaling="banded", factor=2.0),
                dict(scaling="banded", factor=2.0, original_length=100, turns_fast=1.0, turns_slow=1.0),
                dict(scaling="banded", factor=2.0, original_length=100, turns_slow=0.0)):
        assert status(fn, **dict(dict(rot_dim=128), **bad)) == EINVAL, bad
