"""Host-side checks of the 4-bit, routing and log-probability calls that need no GPU: argument
errors before any launch, binding refusals, workspace and layout sizes, and the plain
references themselves against closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg
from gemv_dg_bf16_gb300 import _binding as B
from tests import _ref64 as R

P = ctypes.c_void_p
A, U = 0x10000, 0x10002                  # fake device addresses: aligned, 2 bytes off


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_dg_bf16_gb300 import build
    build.build()
    return dg.lib()


def test_fp4_argument_errors():
    L = dg.lib()
    for f in (L.dg_quant_fp4_blockscale, L.dg_dequant_fp4_blockscale):
        deq = f is L.dg_dequant_fp4_blockscale
        call = lambda x=A, q=A, s=A, g=0, M=2, K=64, fmt=1: (f(q, s, g or None, x, M, K, fmt, None) if deq
                                                             else f(x, q, s, g or None, M, K, fmt, None))
        assert call(x=0) == 1 and call(q=0) == 1 and call(s=0) == 1
        assert call(M=0) == 1 and call(K=0) == 1 and call(fmt=2) == 1 and call(fmt=-1) == 1
        assert call(fmt=0, g=A) == 1
        assert call(K=48) == 3
        assert call(x=U) == 2 and call(q=U) == 2 and call(s=U) == 2 and call(g=U) == 2
    call = lambda x=A, W=A, s=A, gx=0, gw=0, y=A, M=2, N=64, K=256, fmt=1, ws=A, wsb=1 << 20: \
        L.dg_gemv_a4w4_blockscale(x, W, s, gx or None, gw or None, y, M, N, K, fmt, ws, wsb, None, None)
    assert call(M=0) == 1 and call(M=513) == 1 and call(N=0) == 1 and call(fmt=3) == 1
    assert call(K=264) == 3
    assert call(s=0) == 1 and call(W=U) == 2 and call(y=U) == 2 and call(ws=0) == 1 and call(ws=U) == 2
    assert call(fmt=0, gx=A) == 1 and call(fmt=0, gw=A) == 1 and call(gw=U) == 2
    assert call(wsb=32768) == 4


def test_fp4_sizes():
    for fmt, b in ((0, 32), (1, 16)):
        for rows, K in ((1, 32), (128, 64), (129, 4096), (300, 1056)):
            nb = K // b
            want = -(-rows // 128) * -(-nb // 4) * 512
            assert dg.dg_fp4_scale_bytes(rows, K, fmt) == want == int(np.prod(dg.fp4_scale_shape(rows, K, fmt)))
    assert dg.dg_fp4_scale_bytes(0, 32, 0) == dg.dg_fp4_scale_bytes(1, 48, 0) == dg.dg_fp4_scale_bytes(1, 32, 2) == 0
    w = dg.dg_workspace_bytes(dg.DG_OP_GEMV_A4W4, 512, 64, 4096)
    assert w >= 32768 + 512 * 2048 + 4 * 64 * 512


def test_a4w4_select_and_table(tmp_path):
    import json
    for M in (1, 16, 100, 300, 512):
        c = dg.dg_select(dg.DG_OP_GEMV_A4W4, M, 4096, 4096)
        assert c.variant == dg.DG_VAR_TC and c.params[1] == 0
    dg.dg_set_numerics(dg.DG_NUMERICS_BATCH_INVARIANT)
    try:
        assert {dg.dg_select(dg.DG_OP_GEMV_A4W4, M, 4096, 4096).as_tuple()[1][1] for M in (1, 200, 512)} == {1}
    finally:
        dg.dg_set_numerics(dg.DG_NUMERICS_FASTEST)

    def check(pick):
        doc = {"format": "libdecodegemm-table",
               "identity": {"arch": "sm_103", "driver": 13000, "runtime": 13000, "build": dg.dg_build_id(),
                            "selection_space": dg.dg_selection_space()},
               "entries": [{"op": "gemv_a4w4", "M": 4, "N": 64, "K": 64, "pick": pick}]}
        p = tmp_path / "t.json"
        p.write_text(json.dumps(doc))
        return dg.dg_table_check(str(p), "sm_103", 13000, 13000)
    assert check({"variant": 3, "params": [4, 1]})[0] == 0
    assert check({"variant": 1, "params": [4, 8]})[0] == 6 and "tensor cores only" in check({"variant": 1, "params": [4, 8]})[2]
    assert check({"variant": 3, "params": [4, 2]})[0] == 6
    assert B._OP_NAMES[dg.DG_OP_GEMV_A4W4] == "gemv_a4w4"


def test_route_argument_errors():
    L = dg.lib()

    def call(x=A, kind=1, ld=64, bias=0, ids=A, w=A, M=2, E=64, prm=None, **kw):
        p = dict(topk=4, n_group=1, topk_group=1, group_top=1, score=0, renorm=1, scale=1.0)
        p.update(kw)
        return L.dg_moe_route(x, kind, ld, bias or None, prm or B.RouteParams(**p), ids, w, M, E, None)
    assert call(x=0) == 1 and call(ids=0) == 1 and call(w=0) == 1 and call(M=0) == 1 and call(E=0) == 1
    assert call(kind=2) == 1 and call(ld=63) == 1
    assert call(x=U) == 2 and call(x=A + 1, kind=0) == 2 and call(bias=U) == 2 and call(ids=U) == 2 and call(w=A + 1) == 2
    for kw in (dict(topk=0), dict(n_group=0), dict(topk_group=0), dict(topk_group=2), dict(group_top=0), dict(group_top=3),
               dict(score=2), dict(renorm=2)):
        assert call(**kw) == 1, kw
    for kw in (dict(E=1025, ld=1025), dict(topk=33), dict(n_group=3, topk_group=3), dict(n_group=64, topk_group=64, topk=1),
               dict(n_group=32, topk_group=1, topk=3)):
        assert call(**kw) == 3, kw
    assert L.dg_moe_route(A, 1, 64, None, None, A, A, 2, 64, None) == 1


def test_logprobs_argument_errors():
    L = dg.lib()
    call = lambda x=A, kind=0, ld=64, tok=A, scale=1.0, n=2, lp=A, rk=A, en=A, ti=A, tl=A, M=2, V=64: L.dg_logprobs(
        x, kind, ld, tok or None, scale, n, lp or None, rk or None, en or None, ti or None, tl or None, M, V, None)
    assert call(x=0) == 1 and call(M=0) == 1 and call(V=0) == 1 and call(kind=5) == 1 and call(ld=60) == 1
    assert call(scale=0.0) == 1 and call(scale=-1.0) == 1 and call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(n=-1) == 1 and call(n=0) == 1 and call(ti=0) == 1 and call(tl=0) == 1 and call(tok=0) == 1
    assert call(n=33) == 3
    assert call(x=A + 1) == 2 and call(x=U, kind=1) == 2 and call(tok=A + 4) == 2 and call(lp=U) == 2 and call(ti=U) == 2


def test_binding_refuses_mismatched_tensors():
    bf, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
    z = lambda shape, t: torch.zeros(shape, dtype=t)
    x = z((2, 64), bf)
    sh = dg.fp4_scale_shape
    cases = [
        (lambda: dg.dg_quant_fp4_blockscale(x, 2), "fmt"),
        (lambda: dg.dg_quant_fp4_blockscale(z((2, 64), f32), 1), "x: dtype"),
        (lambda: dg.dg_quant_fp4_blockscale(x, 1), "x: tensors must be contiguous CUDA"),
        (lambda: dg.dg_dequant_fp4_blockscale(z((2, 32), bf), z(sh(2, 64, 1), u8), 1), "q: dtype"),
        (lambda: dg.dg_gemv_a4w4_blockscale(x, z((8, 31), u8), z(sh(8, 64, 1), u8), 1, ws=z((9,), u8)), "x: tensors"),
        (lambda: dg.dg_moe_route(z((2, 8), torch.float16), 2), "logits: dtype"),
        (lambda: dg.dg_moe_route(z((8,), f32), 2), "logits: shape"),
        (lambda: dg.dg_moe_route(z((2, 8), f32), 2), "logits: rows"),
        (lambda: dg.dg_logprobs(z((2, 8), i32)), "logits: dtype"),
    ]
    for fn, needle in cases:
        with pytest.raises(ValueError) as e:
            fn()
        assert needle in str(e.value), (needle, str(e.value))


def test_constants_match_header():
    import os
    import re
    from tests._helpers import ROOT
    hdr = open(os.path.join(ROOT, "include", "dg.h")).read()
    d = dict((k, int(v)) for k, v in re.findall(r"#define\s+(DG_(?:FP4|LOGITS|SCORE)_\w+)\s+(\d+)", hdr))
    assert len(d) == 6
    for k, v in d.items():
        assert getattr(dg, k) == v, k


# ---------------------------------------------------------------- the references themselves

def test_reference_e2m1_and_e4m3_rounding():
    pts = {0.0: 0, 0.25: 0, 0.2500001: 1, 0.5: 1, 0.75: 2, 0.7499999: 1, 1.25: 2, 1.2500001: 3, 1.75: 4, 2.5: 4,
           2.5000002: 5, 3.5: 6, 3.4999998: 5, 5.0: 6, 5.0000005: 7, 6.0: 7, 900.0: 7}
    for v, c in pts.items():
        assert R.nearest_even(np.array([np.float32(v)]), R.E2M1)[0] == c, v
    t = torch.linspace(0, 500, 100001)
    want = t.clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.nearest_even(t.numpy(), R.e4m3_table()), want)
    assert np.array_equal(R.e4m3_table().astype(np.float32),
                          torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy())


def test_reference_quant_closed_forms():
    x = np.zeros((2, 64), np.float32)
    x[0, :8] = [6, -4, 3, 2, 1.5, 1, 0.5, 0]          # amax 6: MX scale 1 (byte 127), codes are the values
    x[1, 0] = 7.5                                     # MX: e = 2 - 2 = 0, saturates at 6
    code, byte = R.fp4_quant(x, 0)
    assert byte[0, 0] == 127 and code[0, :8].tolist() == [7, 14, 5, 4, 3, 2, 1, 0] and byte[1, 0] == 127 and code[1, 0] == 7
    assert byte[0, 1] == 0 and (code[0, 32:] == 0).all()
    code, byte = R.fp4_quant(x, 1)
    assert byte[0, 0] == 0x38 and code[0, :8].tolist() == [7, 14, 5, 4, 3, 2, 1, 0]      # s = 1
    code, byte = R.fp4_quant(x, 1, 0.5)
    assert byte[0, 0] == 0x40 and code[0, 0] == 7                                        # s = 2
    q = R.pack(code)
    assert np.array_equal(R.unpack(q), code) and q[0, 0] == (code[0, 0] | code[0, 1] << 4)
    t = R.tile(np.arange(300 * 5, dtype=np.int64).reshape(300, 5).astype(np.uint8))
    assert t.shape == (3, 2, 512) and t[1, 1, (140 % 32) * 16 + 0 * 4 + 0] == (140 * 5 + 4) % 256


def test_reference_route_and_logprobs_closed_forms():
    ids, w, _ = R.route(np.array([[0.0, np.log(3.0), 0.0, -np.inf]]), 3, False)
    assert ids[0].tolist() == [1, 0, 2] and np.allclose(w[0], [0.6, 0.2, 0.2])
    ids, w, _ = R.route(np.array([[0.0, 1.0, 2.0, 3.0]]), 1, True, bias=np.array([9.0, 0, 0, 0]), renorm=False)
    assert ids[0, 0] == 0 and abs(w[0, 0] - 0.5) < 1e-15                                 # bias moves the pick only
    ids, _, _ = R.route(np.array([[5.0, 0, 4.0, 4.0]]), 1, True, n_group=2, topk_group=1, group_top=2)
    assert ids[0, 0] == 2                                                                # the pair beats the single
    r = R.logprobs(np.zeros((1, 8)), np.array([3]), 2)
    assert abs(r["logprob"][0] + np.log(8)) < 1e-12 and abs(r["entropy"][0] - np.log(8)) < 1e-12
    assert r["rank"][0] == 0 and r["top_ids"][0].tolist() == [0, 1]
    r = R.logprobs(np.array([[np.log(0.7), np.log(0.2), np.log(0.1), -np.inf]]), np.array([1]), 5)
    assert np.allclose(np.exp(r["logprob"]), 0.2) and r["rank"][0] == 1 and r["top_ids"][0].tolist() == [0, 1, 2, -1, -1]
    far = R.logprobs(np.full((1, 50), -5.0e29), np.array([3]), 1)
    assert abs(far["entropy"][0] - np.log(50)) < 1e-12 and abs(far["logprob"][0] + np.log(50)) < 1e-12
    assert abs(r["entropy"][0] + 0.7 * np.log(0.7) + 0.2 * np.log(0.2) + 0.1 * np.log(0.1)) < 1e-12
