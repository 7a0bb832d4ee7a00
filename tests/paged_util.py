"""Plain 64-bit forms of the rotation, the append and the attention over a
paged cache, and the error bounds the GPU results are held to.

Rounding to a type of unit roundoff u (half its eps: bf16 2^-8, f16 2^-11, f32
2^-24) moves a value by at most u times its size; every bound below counts such
roundings, in 64 bits, from the data.
"""
from __future__ import annotations

import math

import numpy as np
import torch

TORCH_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U32 = 2.0 ** -24


def unit(dtype: str) -> float:
    return torch.finfo(TORCH_DT[dtype]).eps / 2


# ---------------------------------------------------------------- rotation ---
def rope64(x, positions, inv_freq, rot, layout, magnitude=1.0):
    """x [T, H, D] float64; the definition, pair by pair."""
    x = x.double()
    y = x.clone()
    a = positions.double()[:, None] * inv_freq.double()[None]          # [T, rot / 2]
    c, s = (magnitude * a.cos())[:, None], (magnitude * a.sin())[:, None]
    i = torch.arange(rot // 2)
    u, w = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    y[..., u] = x[..., u] * c - x[..., w] * s
    y[..., w] = x[..., u] * s + x[..., w] * c
    return y


def rope_tol(x, ref, dtype, rot, magnitude=1.0):
    """One rounding of the result; before it, on the pair's size (at most
    |u| + |w| <= 2 max|x|): the fp32 angle fraction is off by 2^-26 turns (2^-25
    relative of at most half a turn) = 1e-7, cos and sin by 2 units, their
    products with the magnitude, the two products and the sum by one each."""
    big = 2 * x.abs().amax(-1, keepdim=True).double() * magnitude
    return unit(dtype) * ref.abs() * (1 + 1e-6) + big * (2 * math.pi * 2.0 ** -26 + 6 * U32)


# --------------------------------------------------------------- batches ----
class Batch:
    """A batch on a paged cache (host tensors): `new` tokens and `kv` keys of
    each sequence, pages in random order, whatever is unused filled with
    `junk`."""

    def __init__(self, new, kv, Hq, Hkv, D, page, dtype, seed=0, order="pthd", lead=0, tail=0, junk=float("nan"),
                 q_gain=2.0):
        g = torch.Generator().manual_seed(seed)
        dt = TORCH_DT[dtype]
        self.new, self.kv, self.Hq, self.Hkv, self.D, self.page, self.dtype, self.order = (
            list(new), list(kv), Hq, Hkv, D, page, dtype, order)
        self.lead, self.tail = lead, tail
        self.T = lead + sum(new) + tail
        need = [(max(n, 0) + page - 1) // page for n in kv]
        self.n_pages = sum(need) + 3
        self.max_pages = max(need + [1]) + 1
        ids = torch.randperm(self.n_pages, generator=g)[:sum(need)]
        self.table = torch.full((len(self.new), self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n].int()
            at += n
        self.starts = torch.tensor(np.cumsum([lead] + self.new), dtype=torch.int32)
        self.lens = torch.tensor(self.kv, dtype=torch.int32)
        # [page, token, head, dim], junk wherever no sequence has a key
        self.k = torch.full((self.n_pages, page, Hkv, D), junk, dtype=dt)
        self.v = torch.full((self.n_pages, page, Hkv, D), junk, dtype=dt)
        self.keys = [torch.randn(n, Hkv, D, generator=g).to(dt) for n in self.kv]
        self.vals = [torch.randn(n, Hkv, D, generator=g).to(dt) for n in self.kv]
        for b, n in enumerate(self.kv):
            self.store(b, self.keys[b], self.vals[b])
        self.q = (q_gain * torch.randn(self.T, Hq, D, generator=g)).to(dt)

    def store(self, b, keys, vals):
        for j in range(keys.shape[0]):
            p = int(self.table[b, j // self.page])
            self.k[p, j % self.page], self.v[p, j % self.page] = keys[j], vals[j]

    def cache(self, t):
        """The cache in its storage order, on the device, and its strides."""
        t = t if self.order == "pthd" else t.transpose(1, 2).contiguous()
        return t.cuda()

    @property
    def strides(self):
        p, h, d = self.page, self.Hkv, self.D
        return (p * h * d, h * d, d) if self.order == "pthd" else (p * h * d, d, p * d)

    def read(self, t):
        """A device cache back as [page, token, head, dim] on the host."""
        t = t.cpu()
        return t if self.order == "pthd" else t.transpose(1, 2)


# --------------------------------------------------------------- attention ---
def attention64(bt: Batch, scale=None, causal=True, window=0, cap=0.0, slopes=None):
    """(out, lse, tolerance of out, tolerance of lse), rows outside the batch
    NaN."""
    scale = 1.0 / math.sqrt(bt.D) if scale is None else scale
    G = bt.Hq // bt.Hkv
    nan = float("nan")
    out = torch.full((bt.T, bt.Hq, bt.D), nan, dtype=torch.float64)
    lse = torch.full((bt.T, bt.Hq), nan, dtype=torch.float64)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for b, (n, m) in enumerate(zip(bt.new, bt.kv)):
        t0 = int(bt.starts[b])
        pos = torch.arange(m - n, m)
        away = torch.arange(m)[None, :] - pos[:, None]                   # [n, m]
        seen = torch.ones(n, m, dtype=torch.bool)
        if causal:
            seen &= away <= 0
        if window:
            seen &= away > -window
        for h in range(bt.Hq):
            q = bt.q[t0:t0 + n, h].double()
            k, v = bt.keys[b][:, h // G].double(), bt.vals[b][:, h // G].double()
            # a key no row may see takes no part, whatever it holds
            kz = torch.where(torch.isfinite(k), k, torch.zeros_like(k))
            s = q @ kz.T * scale
            s = torch.where(torch.isfinite(k).all(1)[None, :], s, torch.full_like(s, nan))
            # a product's error: D + 2 roundings of its terms, the scale's and the sum's
            ds = (bt.D + 4) * U32 * (q.abs() @ kz.abs().T) * scale
            if cap:
                s = cap * torch.tanh(s / cap)
                ds = ds + 8 * U32 * cap
            if slopes is not None:
                s = s + float(slopes[h]) * away
                ds = ds + 2 * U32 * (float(slopes[h]) * away).abs()
            ds = ds + 4 * U32 * s.abs()
            s = s.masked_fill(~seen, -math.inf)
            top = s.amax(1, keepdim=True) if m else torch.full((n, 1), -math.inf, dtype=torch.float64)
            base = torch.where(top == -math.inf, torch.zeros_like(top), top)
            p = torch.where(seen, torch.exp(s - base), torch.zeros_like(s))
            l = p.sum(1, keepdim=True)
            empty = (l == 0).squeeze(1)
            w = torch.where(l > 0, p / l, torch.where(torch.isnan(l), l, torch.zeros_like(p)))
            vz = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
            o = w @ vz
            # a non-finite value reaches exactly the rows that see its key
            for j in torch.nonzero(~torch.isfinite(v).all(1)).flatten().tolist():
                rows = seen[:, j]
                o[rows] = o[rows] + torch.where(torch.isfinite(v[j]), torch.zeros_like(v[j]), v[j])[None]
            out[t0:t0 + n, h] = o
            lse[t0:t0 + n, h] = torch.where(empty, torch.full_like(l[:, 0], -math.inf), base[:, 0] + torch.log(l[:, 0]))
            d = torch.where(seen, ds, torch.zeros_like(ds)).amax(1, keepdim=True) if m else torch.zeros(n, 1)
            a = w.abs() @ vz.abs()
            cnt = seen.sum(1, keepdim=True).double()
            # weights off by e^(2 d) and the exponential's 2 units; sums of cnt
            # terms, each partial sum rescaled: 2 roundings a term at most
            rel = 2 * d + (8 + 2 * cnt) * U32
            u = unit(bt.dtype)
            tol[t0:t0 + n, h] = u * o.abs() + (u if bt.dtype != "f32" else 0.0) * a * (1 + u) + rel * a * 1.01
            tol_l[t0:t0 + n, h] = (d + (8 + 2 * cnt) * U32).squeeze(1) + 2 * U32 * lse[t0:t0 + n, h].abs().nan_to_num(0, 0, 0)
    return out, lse, tol, tol_l


def wide_table(bt: Batch):
    """The page table with so many (unused) columns that the call is taken for
    one over long sequences: many query rows then run on the kernel for them,
    which short calls leave to the one for few."""
    units = len(bt.new) * bt.Hkv
    cols = max(bt.max_pages, -(-4000 * 64 // (bt.page * units)) + 1)
    t = torch.full((len(bt.new), cols), -1, dtype=torch.int32)
    t[:, :bt.max_pages] = bt.table
    return t


def run_attention(q, bt: Batch, workspace=None, max_q_len=None, lse=True, k=None, v=None, q_strided=False, stream=None,
                  wide=False, **kw):
    dt = TORCH_DT[bt.dtype]
    fill = 7.0
    if q_strided:                     # the query heads inside a fused [Q | K | V] row
        wide = (bt.Hq + 2 * bt.Hkv) * bt.D
        buf = torch.full((bt.T, wide), float("nan"), dtype=dt)
        buf[:, :bt.Hq * bt.D] = bt.q.reshape(bt.T, -1)
        qd, qs = buf.cuda(), (wide, bt.D)
    else:
        qd, qs = bt.q.cuda(), None
    out = torch.full((bt.T, bt.Hq, bt.D), fill, dtype=dt, device="cuda")
    ls = torch.full((bt.T, bt.Hq), fill, dtype=torch.float32, device="cuda") if lse else None
    slopes = kw.pop("slopes", None)
    sl = None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda")
    table = wide_table(bt) if wide else bt.table
    keep = [bt.cache(bt.k) if k is None else k, bt.cache(bt.v) if v is None else v, table.cuda(), bt.starts.cuda(),
            bt.lens.cuda()]
    q.qmv_paged_attention(qd, *keep, out, ls, bt.T, bt.Hq, bt.Hkv, bt.D, len(bt.new), bt.n_pages, bt.page,
                          table.shape[1], kw.pop("scale", 1.0 / math.sqrt(bt.D)), bt.dtype, slopes=sl,
                          max_q_len=(max(bt.new) if bt.new else 0) if max_q_len is None else max_q_len, cache_strides=bt.strides,
                          q_strides=qs, workspace=workspace, softcap=kw.pop("cap", 0.0), stream=stream, **kw)
    torch.cuda.synchronize()
    return out, ls


def check_attention(bt: Batch, out, lse, ref, fill=7.0):
    o, l, tol, tol_l = ref
    out = out.double().cpu()
    rows = ~torch.isnan(l).all(1) if l.numel() else torch.zeros(0, dtype=torch.bool)
    inside = torch.zeros(bt.T, dtype=torch.bool)
    inside[bt.lead:bt.lead + sum(bt.new)] = True
    assert (out[~inside] == fill).all(), "rows outside the batch were written"
    same = (out == o) | (torch.isnan(out) & torch.isnan(o)) | ((out - o).abs() <= tol)
    same = same[inside]
    worst = ((out - o).abs() / tol.clamp_min(1e-300))[inside]
    assert same.all(), (f"{int((~same).sum())} of {same.numel()} outputs, worst {worst.nan_to_num(1e9).max():.3g} x the "
                        f"bound, first at {torch.nonzero(~same)[0].tolist()}")
    if lse is not None:
        lse = lse.double().cpu()
        assert (lse[~inside] == fill).all()
        ok = (lse == l) | (torch.isnan(lse) & torch.isnan(l)) | ((lse - l).abs() <= tol_l)
        assert ok[inside].all(), f"lse off by {(lse - l).abs()[inside].nan_to_num(1e9).max()}"
    return rows
