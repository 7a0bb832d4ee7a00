"""The attention half of a decode layer, as a user runs it: Q / K / V projection,
rotation and append to the paged cache, attention over it, output projection,
token after token, eager and captured into one graph that is replayed."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from gpu_util import THREADS, compare, require_cuda, to_f64
from paged_util import Batch, attention64, rope64, rope_tol

pytestmark = pytest.mark.gpu

HQ, HKV, D, K, G, PAGE = 8, 2, 64, 512, 64, 16
NQ, NKV = HQ * D, HKV * D


@pytest.fixture(scope="module")
def q():
    return require_cuda()


class Layer:
    def __init__(self, q, past, seed=0):
        self.q, self.B = q, len(past)
        self.host = []
        for i, (n, k) in enumerate(((NQ, K), (NKV, K), (NKV, K), (K, NQ))):
            g = np.random.default_rng(seed + 10 + i)
            w = torch.tensor(g.normal(size=(n, k)) / np.sqrt(k)).bfloat16().cuda()
            packed = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
            sc = torch.empty(n, k // G, dtype=torch.bfloat16, device="cuda")
            bi = torch.empty_like(sc)
            q.qmv_quantize_affine(w, packed, sc, bi, n, k, 4, G, "bf16")
            self.host.append((packed, sc, bi))
        self.past = list(past)
        need = [(p + 40 + PAGE - 1) // PAGE for p in past]
        self.n_pages, self.max_pages = sum(need) + 1, max(need)
        ids = torch.randperm(self.n_pages, generator=torch.Generator().manual_seed(seed))[:sum(need)]
        self.table = torch.zeros(self.B, self.max_pages, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n].int()
            at += n
        g = torch.Generator().manual_seed(seed + 1)
        self.keys = [torch.randn(p, HKV, D, generator=g).bfloat16() for p in past]
        self.vals = [torch.randn(p, HKV, D, generator=g).bfloat16() for p in past]
        kc = torch.zeros(self.n_pages, PAGE, HKV, D, dtype=torch.bfloat16)
        vc = torch.zeros_like(kc)
        for b in range(self.B):
            for j in range(past[b]):
                p = int(self.table[b, j // PAGE])
                kc[p, j % PAGE], vc[p, j % PAGE] = self.keys[b][j], self.vals[b][j]
        f, m = q.qmv_rope_frequencies(D)
        self.f = torch.tensor(f, dtype=torch.float32)
        self.d = dict(k=kc.cuda(), v=vc.cuda(), table=self.table.cuda(), f=self.f.cuda(),
                      starts=torch.arange(self.B + 1, dtype=torch.int32, device="cuda"),
                      lens=torch.tensor(past, dtype=torch.int32, device="cuda"),
                      x=torch.empty(self.B, K, dtype=torch.bfloat16, device="cuda"),
                      qkv=torch.empty(self.B, NQ + 2 * NKV, dtype=torch.bfloat16, device="cuda"),
                      qr=torch.empty(self.B, HQ, D, dtype=torch.bfloat16, device="cuda"),
                      att=torch.empty(self.B, HQ, D, dtype=torch.bfloat16, device="cuda"),
                      y=torch.empty(self.B, K, dtype=torch.bfloat16, device="cuda"),
                      ws=torch.zeros(q.PAGED_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda"))

    def step(self):
        q, d, B = self.q, self.d, self.B
        d["lens"].add_(1)
        wq, wk, wv, wo = self.host
        q.qmv_affine_qkv(d["x"], wq, wk, wv, d["qkv"], B, NQ, NKV, K, 4, G, "bf16")
        q.qmv_kv_append(d["qkv"], d["k"], d["v"], d["table"], d["starts"], d["lens"], d["f"], d["qr"], B, HQ, HKV, D, D,
                        "half", B, self.n_pages, PAGE, self.max_pages, "bf16")
        q.qmv_paged_attention(d["qr"], d["k"], d["v"], d["table"], d["starts"], d["lens"], d["att"], None, B, HQ, HKV, D,
                              B, self.n_pages, PAGE, self.max_pages, D ** -0.5, "bf16", max_q_len=1, workspace=d["ws"])
        q.qmv_affine(d["att"], *wo, d["y"], B, K, NQ, 4, G, "bf16")

    def check(self):
        """Every stage against the definition, from the stage before's own output."""
        d, B = {k: v.cpu() for k, v in self.d.items()}, self.B
        rows = d["qkv"].view(B, HQ + 2 * HKV, D)
        pos = torch.tensor(self.past)
        turned = rope64(rows, pos, self.f, D, "half")
        tol = rope_tol(rows, turned, "bf16", D)
        assert ((d["qr"].double() - turned[:, :HQ]).abs() <= tol[:, :HQ]).all()
        bt = Batch([1] * B, [p + 1 for p in self.past], HQ, HKV, D, PAGE, "bf16")
        for b in range(B):
            j = self.past[b]
            p = int(self.table[b, j // PAGE])
            assert ((d["k"][p, j % PAGE].double() - turned[b, HQ:HQ + HKV]).abs() <= tol[b, HQ:HQ + HKV]).all()
            assert torch.equal(d["v"][p, j % PAGE], rows[b, HQ + HKV:])
            self.keys[b] = torch.cat([self.keys[b], d["k"][p, j % PAGE][None]])
            self.vals[b] = torch.cat([self.vals[b], d["v"][p, j % PAGE][None]])
            self.past[b] += 1
        bt.keys, bt.vals, bt.q = self.keys, self.vals, d["qr"]
        out, _, otol, _ = attention64(bt)
        assert ((d["att"].double() - out).abs() <= otol).all()
        wo = [t.cpu() for t in self.host[3]]
        as_np = lambda t: t.contiguous().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
        ref, ad = oracle.qmv_affine(as_np(d["att"]).reshape(B, NQ), wo[0].numpy(), as_np(wo[1]), as_np(wo[2]), B, K, NQ, 4, G,
                                    "bf16", threads=THREADS)
        compare(to_f64(d["y"]), ref, ad, "bf16", what="output projection")


@pytest.mark.parametrize("past", [[0], [5, 300, 15], [31, 0, 64, 1000, 16, 7, 128, 2]])
def test_tokens_in_turn(q, past):
    layer = Layer(q, past)
    g = torch.Generator().manual_seed(9)
    for _ in range(3):
        layer.d["x"].copy_(torch.randn(layer.B, K, generator=g))
        layer.step()
        torch.cuda.synchronize()
        layer.check()


def test_captured_and_replayed(q):
    layer = Layer(q, [12, 130])
    g = torch.Generator().manual_seed(3)
    layer.step()                                   # kernels are loaded before the capture
    torch.cuda.synchronize()
    layer.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    for _ in range(4):
        layer.d["x"].copy_(torch.randn(2, K, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        layer.check()
