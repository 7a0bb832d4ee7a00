"""QMV_PDL=0 turns programmatic dependent launch off for the rotation, the append
and the attention too: the dependencies of a captured chain of them say which."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

from gpu_util import require_cuda

pytestmark = pytest.mark.gpu

CODE = '''
import ctypes, torch, weight_quantized_matrix_b200 as q
rt = ctypes.CDLL("libcudart.so.12")             # torch's, loaded already
i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
kinds = []
for dt, name, T, wide, shift in ((torch.bfloat16, "bf16", 1, 13, 0), (torch.bfloat16, "bf16", 200, 40000, 0),
                                 (torch.float32, "f32", 3, 13, 0), (torch.bfloat16, "bf16", 2, 13, 1)):
    x = torch.randn(T, 8 * 64, device="cuda").to(dt)
    k, v = (torch.zeros(20 * 16 * 2 * 64 + shift, device="cuda", dtype=dt)[shift:] for _ in range(2))
    table = torch.zeros(1, wide, dtype=torch.int32, device="cuda")
    table[0, :13] = torch.arange(13, device="cuda")
    starts, lens, f, pos = i32(0, T), i32(T), torch.ones(32, device="cuda"), torch.arange(T, device="cuda").int()
    y, qr, out = (torch.empty(T, n, 64, device="cuda", dtype=dt) for n in (8, 4, 4))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        q.qmv_rope(x, y, pos, f, T, 8, 64, 64, "half", name)
        q.qmv_kv_append(y, k, v, table, starts, lens, f, qr, T, 4, 2, 64, 64, "half", 1, 20, 16, wide, name)
        q.qmv_paged_attention(qr, k, v, table, starts, lens, out, None, T, 4, 2, 64, 1, 20, 16, wide, 0.125, name)
        q.qmv_rope(out, qr, pos, f, T, 4, 64, 64, "half", name)
    n = ctypes.c_size_t(3)
    ends, data = [(ctypes.c_void_p * 3)() for _ in range(2)], (ctypes.c_ubyte * 24)()
    assert rt.cudaGraphGetEdges_v2(ctypes.c_void_p(g.raw_cuda_graph()), *ends, data, ctypes.byref(n)) == 0 and n.value == 3
    kinds += data[2::8]                         # the third byte of an edge's 8: 0 full, 1 programmatic
print("KINDS", *kinds)
'''


@pytest.mark.parametrize("value,want", [(None, 1), ("0", 0), ("1", 1)])
def test_dependencies_of_a_captured_chain(value, want):
    require_cuda()
    env = {k: v for k, v in os.environ.items() if k != "QMV_PDL"}
    if value is not None:
        env["QMV_PDL"] = value
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stderr[-2000:]
    kinds = r.stdout.split("KINDS")[1].split()
    assert kinds == [str(want)] * 12, kinds
