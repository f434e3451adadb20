"""The benchmark's one JSON line (no GPU): rows as columns, without loss, in a line that fits the
16 KB that a harness may keep of it."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402


def _rows(op, n, **more):
    return [dict(op=op, M=128, N=248320, K=12288, **more, us=1234.567 + i, gbs=6789.1, frac=0.9876, weight_bytes=1017118724)
            for i in range(n)]


def test_columns_hold_every_value():
    rows = _rows("gemv_bf16", 3)
    rows[1]["tflops"] = 12.5
    t = json.loads(json.dumps(bench._columns(rows)))
    back = [{k: v for k, v in zip(t["cols"], r) if v is not None} for r in t["rows"]]
    assert back == [{k: v for k, v in r.items() if k != "op"} for r in rows]
    assert bench._columns([]) == {"cols": [], "rows": []}


def test_line_of_every_table_is_short():
    """As many rows as the default run reports, at their widest."""
    ops = {"gate_up_silu": 11, "head_fp8_argmax": 5, "moe_w1_silu": 5, "moe_w2": 5, "gemv_mid_m": 12, "gemv_a8w8": 14,
           "gemv_bf16_invariant": 20, "chain_mlp": 5, "chain_moe": 5}
    res = {"shapes": bench._columns(_rows("gemv_bf16", 40)),
           "ops": {k: bench._columns(_rows(k, n, tflops_per_call=0.012885, parts_us=1234.567)) for k, n in ops.items()},
           "cold": [1234.567] * 40}
    # (the contract's own keys take another 3 KB)
    assert len(json.dumps(res, separators=(",", ":"))) < 13 * 1024
