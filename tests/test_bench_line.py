"""bench.py's result line stays short enough to be read back: the breakdown's lines
are shortened in it, nothing of their shape, time or fraction lost."""
from __future__ import annotations

import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_short_lines():
    sys.path.insert(0, ROOT)
    import bench
    plan = "path=tcf chunk=128 maxm=1 rows_per_warp=1 warps_k=4 warps_rows=2 tile_iters=32 grid=128 block=288 " * 2
    lines = [{"set": bench.SHAPE_SETS[i % len(bench.SHAPE_SETS)], "shape": f"affine b6 g128 bf16 M={i} N=K=16384", "us_per_call": 7.3 + i,
              "us_p5": 7.2, "us_p95": 7.4, "GB_s": 1792.0, "frac_of_hbm": 0.2775, "calls_per_graph": 21, "plan": plan}
             for i in range(130)]
    short = bench.short_lines(lines)
    assert len(json.dumps(short)) < 12000 < len(json.dumps(lines))
    back = [(k, *row) for k in short for row in short[k]]
    assert sorted(back) == sorted((x["set"], x["shape"], x["us_per_call"], x["frac_of_hbm"]) for x in lines)
