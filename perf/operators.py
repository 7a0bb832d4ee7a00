"""Measured cases of the operators between a decode layer's Q/K/V projection and
its output projection: the rotary rotation, the append of rotated keys and of
values to a paged cache, and attention over that cache.

`run` gives the plain form (elementary torch operations in fp32, the rotation's
angles in fp64) or, with `own` set, the calls a user makes of the library.  Head
layouts follow the 4096-wide decode layer of this repository (32 query heads
and 8 key / value heads of 128) and generic neighbours of it.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2}
# the attention call's workspace, zeroed once and kept by the user's program
_WORKSPACE = 40 << 20


# ------------------------------------------------------------------ cases ---
def _rope(name, T, H, D, rot, layout, dtype, far, stretch=1.0):
    c = {"op": "rope", "T": T, "H": H, "D": D, "rot": rot, "layout": layout, "dtype": dtype, "far": far,
         "stretch": stretch}
    return {"name": name, **c} if name else c


def _batch(op, name, seqs, new, past, heads, kv_heads, D, page, dtype, order, lens, **more):
    c = {"op": op, "seqs": seqs, "new_lo": new[0], "new_hi": new[1], "past_lo": past[0], "past_hi": past[1],
         "Hq": heads, "Hkv": kv_heads, "D": D, "page": page, "dtype": dtype, "order": order, "lens": lens, **more}
    return {"name": name, **c} if name else c


def _append(name, *a, rot, layout):
    return _batch("append", name, *a, rot=rot, layout=layout)


def _attn(name, *a, causal=True, window=0, cap=0.0, slopes=False):
    return _batch("attn", name, *a, causal=causal, window=window, cap=cap, slopes=slopes)


def listed():
    return [
        # one token of one request: launch latency
        _rope("rope_token", 1, 40, 128, 128, "half", "bf16", 4096),
        # a long prompt's queries, half of each head rotated, positions past the trained length (stretched angles)
        _rope("rope_prompt", 8192, 32, 128, 64, "interleaved", "f16", 262144, 4.0),
        # a serving step of 64 requests, one token each, from the fused Q/K/V projection's output
        _append("append_step", 64, (1, 1), (0, 4096), 32, 8, 128, 16, "bf16", "pthd", 1, rot=128, layout="half"),
        # prompts of several requests in one call; pages ordered by head first
        _append("append_prompts", 7, (311, 1900), (0, 1000), 32, 8, 128, 64, "bf16", "phtd", 2, rot=128,
                layout="half"),
        # the smallest decode: one token, a short context
        _attn("attn_token_short", 1, (1, 1), (516, 516), 32, 8, 128, 16, "bf16", "pthd", 3),
        # one token of a very long context: the split over the keys
        _attn("attn_token_long", 1, (1, 1), (131000, 131000), 32, 8, 128, 64, "bf16", "pthd", 4),
        # a serving step: 64 requests of ragged lengths
        _attn("attn_step", 64, (1, 1), (300, 8000), 32, 8, 128, 16, "bf16", "phtd", 5),
        # several drafted tokens a request, in fp32, heads of 64, one key head per query head, odd pages
        _attn("attn_drafts_f32", 12, (2, 5), (100, 2100), 16, 16, 64, 24, "f32", "pthd", 6),
        # prompts beside running requests in one call (mixed lengths), a sliding window
        _attn("attn_mixed_window", 24, (1, 700), (0, 6000), 28, 4, 128, 32, "f16", "pthd", 7, window=1024),
        # a prompt chunk whose scores are capped and biased by distance, heads of 64
        _attn("attn_chunk_cap", 2, (1500, 2047), (500, 3001), 32, 8, 64, 16, "bf16", "pthd", 8, cap=30.0,
              slopes=True),
        # a chunk of a long prompt, causal: the matrix products bound it
        _attn("attn_chunk_long", 1, (4096, 4096), (12288, 12288), 32, 8, 128, 64, "bf16", "pthd", 9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    layout = rng.choice(["half", "interleaved"])
    kind = rng.choice(["rope", "append", "append", "decode", "decode", "drafts", "chunk", "chunk"])
    if kind == "rope":
        D = rng.choice([64, 80, 96, 128, 192, 256])
        H = rng.choice([1, 5, 8, 12, 32, 40])
        T = _log(rng, 1, max(2, 8192 * 4096 // (H * D) if H * D > 4096 else 8192))
        return _rope(None, T, H, D, rng.choice([D, D // 2]), layout, dtype, _log(rng, 16, 1000000),
                     rng.choice([1.0, 4.0]))
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
    D = rng.choice([64, 128, 128, 128, 96, 256])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128, 256])
    order = rng.choice(["pthd", "phtd"])
    lens = rng.randrange(1 << 20)
    if kind == "append":
        seqs = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 8192 // seqs))
        return _append(None, seqs, (max(1, hi // 3), hi), (0, 2000), heads, kv_heads, D, page, dtype, order, lens,
                       rot=rng.choice([D, D // 2]), layout=layout)
    window = rng.choice([0, 0, 0, _log(rng, 1, 4000)])
    cap = rng.choice([0.0, 0.0, 30.0])
    slopes = rng.random() < 0.25
    if kind == "decode":
        seqs = _log(rng, 1, 96)
        # keys of one batch: up to a gigabyte of cache
        hi = _log(rng, 16, max(20, (1 << 30) // (2 * kv_heads * D * _ES[dtype]) // seqs))
        hi = min(hi, 200000 // seqs)
        return _attn(None, seqs, (1, 1), (hi // 4, hi), heads, kv_heads, D, page, dtype, order, lens,
                     causal=True, window=window, cap=cap, slopes=slopes)
    if kind == "drafts":
        seqs = _log(rng, 1, 32)
        hi = _log(rng, 16, 60000 // seqs)
        return _attn(None, seqs, (1, rng.choice([3, 5, 8, 17])), (hi // 4, hi), heads, kv_heads, D, page, dtype, order,
                     lens, causal=rng.random() < 0.8, window=window, cap=cap, slopes=slopes)
    seqs = _log(rng, 1, 16)
    most = (4096 if dtype != "f32" else 1000) * 32 // max(32, heads)
    hi = _log(rng, 24, max(25, most // seqs))
    past = _log(rng, 1, max(2, 3 * most // seqs))
    return _attn(None, seqs, (max(1, hi // 5), hi), (0, past), heads, kv_heads, D, page, dtype, order, lens,
                 causal=rng.random() < 0.85, window=window, cap=cap, slopes=slopes)


def _lengths(c):
    """New tokens and cached lengths (new ones included) of each sequence."""
    r = random.Random(c["lens"])
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["seqs"])]
    kv = [n + r.randint(c["past_lo"], c["past_hi"]) for n in new]
    return new, kv


# ----------------------------------------------------------------- inputs ---
def prepare(case, seed):
    c, dev = dict(case), "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DT[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    s = {"case": c}
    if "rot" in c:
        half = torch.arange(c["rot"] // 2, device=dev, dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-2.0 * half / c["rot"]) / c.get("stretch", 1.0)).float()
        s["magnitude"] = 0.1 * math.log(c["stretch"]) + 1.0 if c.get("stretch", 1.0) > 1.0 else 1.0
    if c["op"] == "rope":
        T, H, D = c["T"], c["H"], c["D"]
        s["x"], s["y"] = normal(T, H, D), torch.empty(T, H, D, device=dev, dtype=dt)
        s["positions"] = torch.randint(0, c["far"], (T,), generator=g, device=dev, dtype=torch.int32)
        return s
    new, kv = _lengths(c)
    Hq, Hkv, D, ps = c["Hq"], c["Hkv"], c["D"], c["page"]
    T, wide = sum(new), max((n + ps - 1) // ps for n in kv)
    need = [(n + ps - 1) // ps for n in kv]
    pages = sum(need) + 2
    ids = torch.randperm(pages, generator=g, device=dev).int()
    table = torch.zeros(len(kv), max(wide, 1), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    shape = (pages, ps, Hkv, D) if c["order"] == "pthd" else (pages, Hkv, ps, D)
    s.update(new=new, kv=kv, T=T, table=table, pages=pages, wide=max(wide, 1),
             starts=torch.tensor(starts, dtype=torch.int32, device=dev),
             lens=torch.tensor(kv, dtype=torch.int32, device=dev))
    s["k"], s["v"] = normal(*shape), normal(*shape)
    st = s["k"].stride()
    s["strides"] = (st[0], st[1], st[2]) if c["order"] == "pthd" else (st[0], st[2], st[1])
    if c["op"] == "append":
        s["qkv"] = normal(T, (Hq + 2 * Hkv) * D)
        s["q_out"] = torch.empty(T, Hq, D, device=dev, dtype=dt)
        return s
    # queries of twice the keys' size: softmax weights as uneven as a trained layer's
    s["q"] = (2 * torch.randn(T, Hq, D, generator=g, device=dev)).to(dt)
    s["out"] = torch.empty(T, Hq, D, device=dev, dtype=dt)
    s["lse"] = torch.empty(T, Hq, device=dev, dtype=torch.float32)
    s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=dev, dtype=torch.float32) / Hq) if c["slopes"] else None
    s["workspace"] = torch.zeros(_WORKSPACE, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------ plain forms ---
def _rotate(x, positions, inv_freq, magnitude, layout):
    """x [T, H, D] fp32 rotated by positions [T]; the angles in fp64."""
    r = 2 * inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq.double()
    cos = (angle.cos() * magnitude).float()[:, None]
    sin = (angle.sin() * magnitude).float()[:, None]
    if layout == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _paged(cache, order):
    """The cache as [page, token, head, dim]."""
    return cache if order == "pthd" else cache.transpose(1, 2)


def _token_places(s):
    """Sequence and position of each new token."""
    new = s["starts"][1:] - s["starts"][:-1]
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device=new.device), new, output_size=s["T"])
    i = torch.arange(s["T"], device=new.device) - s["starts"][seq]
    return seq, s["lens"][seq] - new[seq] + i


def _plain_append(s):
    c = s["case"]
    Hq, Hkv, D, ps = c["Hq"], c["Hkv"], c["D"], c["page"]
    seq, pos = _token_places(s)
    x = s["qkv"].view(s["T"], Hq + 2 * Hkv, D)
    turned = _rotate(x[:, :Hq + Hkv].float(), pos, s["inv_freq"], s["magnitude"], c["layout"]).to(x.dtype)
    page, row = s["table"][seq, pos // ps].long(), pos % ps
    _paged(s["k"], c["order"])[page, row] = turned[:, Hq:]
    _paged(s["v"], c["order"])[page, row] = x[:, Hq + Hkv:]
    return turned[:, :Hq], s["k"], s["v"]


def _plain_attention(s):
    c = s["case"]
    B, Hq, Hkv, D, ps = c["seqs"], c["Hq"], c["Hkv"], c["D"], c["page"]
    dev = s["q"].device
    nq, nk = max(s["new"]), max(s["kv"])
    new = s["starts"][1:] - s["starts"][:-1]
    kpos = torch.arange(nk, device=dev)
    page = s["table"][:, kpos // ps].long()
    k = _paged(s["k"], c["order"])[page, kpos % ps].float()                    # [B, nk, Hkv, D]
    v = _paged(s["v"], c["order"])[page, kpos % ps].float()
    i = torch.arange(nq, device=dev)
    token = (s["starts"][:-1, None] + i).clamp(max=s["T"] - 1).long()
    q = s["q"][token].float().view(B, nq, Hkv, Hq // Hkv, D)
    score = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D), k.permute(0, 2, 3, 1))
    score = (score * (1.0 / math.sqrt(D))).view(B, Hq, nq, nk)
    if c["cap"]:
        score = c["cap"] * torch.tanh(score / c["cap"])
    qpos = (s["lens"] - new)[:, None] + i                                       # [B, nq]
    away = kpos - qpos[..., None]                                               # [B, nq, nk]
    if c["slopes"]:
        score = score + s["slopes"][None, :, None, None] * away[:, None].float()
    seen = (kpos < s["lens"][:, None, None]).expand(B, nq, nk)
    if c["causal"]:
        seen = seen & (away <= 0)
    if c["window"]:
        seen = seen & (away > -c["window"])
    score = score.masked_fill(~seen[:, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    score = (score - top).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score.view(B, Hkv, -1, nk), v.transpose(1, 2)).view(B, Hq, nq, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log()).squeeze(-1)
    seq, pos = _token_places(s)
    at = torch.arange(s["T"], device=dev) - s["starts"][seq]
    return o[seq, :, at].to(s["q"].dtype), lse[seq, :, at]


def _plain(s):
    if s["case"]["op"] == "rope":
        return _rotate(s["x"].float(), s["positions"], s["inv_freq"], s["magnitude"], s["case"]["layout"]).to(s["x"].dtype)
    return _plain_append(s) if s["case"]["op"] == "append" else _plain_attention(s)


# -------------------------------------------------------- the library's calls
def _library(s):
    import weight_quantized_matrix_b200 as qmv
    c = s["case"]
    if c["op"] == "rope":
        qmv.qmv_rope(s["x"], s["y"], s["positions"], s["inv_freq"], c["T"], c["H"], c["D"], c["rot"], c["layout"],
                     c["dtype"], magnitude=s["magnitude"])
        return s["y"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "append":
        qmv.qmv_kv_append(s["qkv"], s["k"], s["v"], s["table"], s["starts"], s["lens"], s["inv_freq"], s["q_out"],
                          s["T"], Hq, Hkv, D, c["rot"], c["layout"], c["seqs"], s["pages"], c["page"], s["wide"],
                          c["dtype"], magnitude=s["magnitude"], cache_strides=s["strides"])
        return s["q_out"], s["k"], s["v"]
    qmv.qmv_paged_attention(s["q"], s["k"], s["v"], s["table"], s["starts"], s["lens"], s["out"], s["lse"], s["T"], Hq,
                            Hkv, D, c["seqs"], s["pages"], c["page"], s["wide"], 1.0 / math.sqrt(D), c["dtype"],
                            causal=c["causal"], window=c["window"], softcap=c["cap"], slopes=s["slopes"],
                            max_q_len=max(s["new"]), cache_strides=s["strides"], workspace=s["workspace"])
    return s["out"], s["lse"]


def run(state):
    if own:
        return _library(state)
    return _plain(state)


# ------------------------------------------------------------------- work ---
def work(case):
    c = dict(case)
    es, D = _ES[c["dtype"]], c["D"]
    if c["op"] == "rope":
        n = c["T"] * c["H"]
        return {"bytes": 2 * n * D * es + 4 * c["T"] + 2 * c["rot"], "flops": 3 * n * c["rot"]}
    new, kv = _lengths(c)
    T, Hq, Hkv = sum(new), c["Hq"], c["Hkv"]
    tables = 8 * len(new) + 4 * sum((n + c["page"] - 1) // c["page"] for n in kv)
    if c["op"] == "append":
        return {"bytes": 2 * T * (Hq + 2 * Hkv) * D * es + tables, "flops": 3 * T * (Hq + Hkv) * c["rot"]}
    pairs = keys = 0
    for n, m in zip(new, kv):
        first = m
        for i in range(n):
            p = m - n + i
            hi = min(m, p + 1) if c["causal"] else m
            lo = max(0, p - c["window"] + 1) if c["window"] else 0
            pairs += max(0, hi - lo)
            first = min(first, lo)
        keys += m - first if n else 0
    return {"bytes": 2 * T * Hq * D * es + 4 * T * Hq + 2 * keys * Hkv * D * es + tables, "flops": 4 * D * Hq * pairs}


# ------------------------------------------------- the definition, 64 bits ---
def _turn(x, pos, inv_freq, magnitude, layout):
    """The rotation as a complex product."""
    r = 2 * inv_freq.numel()
    z = torch.polar(torch.full_like(inv_freq.double(), magnitude)[None].expand(pos.numel(), -1).contiguous(),
                    torch.outer(pos.double(), inv_freq.double()))[:, None]
    out = x.clone()
    if layout == "half":
        w = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * z
        out[..., :r // 2], out[..., r // 2:r] = w.real, w.imag
    else:
        w = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * z
        out[..., 0:r:2], out[..., 1:r:2] = w.real, w.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        return _turn(s["x"].double(), s["positions"], s["inv_freq"], s["magnitude"], c["layout"])
    Hq, Hkv, D, ps = c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    if c["op"] == "append":
        k, v, q, at = s["k"].double(), s["v"].double(), [], 0
        kl, vl = (k, v) if c["order"] == "pthd" else (k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3))
        for b, (n, m) in enumerate(zip(s["new"], s["kv"])):
            x = s["qkv"][at:at + n].double().view(n, Hq + 2 * Hkv, D)
            at += n
            pos = torch.arange(m - n, m, device=x.device)
            q.append(_turn(x[:, :Hq], pos, s["inv_freq"], s["magnitude"], c["layout"]))
            turned = _turn(x[:, Hq:Hq + Hkv], pos, s["inv_freq"], s["magnitude"], c["layout"])
            page = s["table"][b].long()[pos // ps]
            kl[page, pos % ps], vl[page, pos % ps] = turned, x[:, Hq + Hkv:]
        return torch.cat(q), k, v
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((s["T"], Hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    at = 0
    for b, (n, m) in enumerate(zip(s["new"], s["kv"])):
        kp = torch.arange(m, device=out.device)
        qp = torch.arange(m - n, m, device=out.device)
        gap = kp[None] - qp[:, None]
        hide = torch.zeros_like(gap, dtype=torch.bool)
        if c["causal"]:
            hide |= gap > 0
        if c["window"]:
            hide |= gap <= -c["window"]
        page, row = s["table"][b].long()[kp // ps], kp % ps
        for h in range(Hq):
            if c["order"] == "pthd":
                k, v = s["k"][page, row, h // G].double(), s["v"][page, row, h // G].double()
            else:
                k, v = s["k"][page, h // G, row].double(), s["v"][page, h // G, row].double()
            z = s["q"][at:at + n, h].double() @ k.T / math.sqrt(D)
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            if c["slopes"]:
                z = z + float(s["slopes"][h]) * gap
            z = z.masked_fill(hide, -math.inf)
            total = torch.logsumexp(z, 1)
            lse[at:at + n, h] = total
            out[at:at + n, h] = torch.where(total[:, None] == -math.inf, 0.0, 1.0) * (
                torch.exp(z - torch.where(total == -math.inf, torch.zeros_like(total), total)[:, None]) @ v)
        at += n
    return out, lse
