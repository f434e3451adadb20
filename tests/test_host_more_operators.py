"""Host-side checks of the 8-bit integer, sorting and logits calls that need no GPU: argument errors before
any launch, binding refusals, sizes, table rules, and the plain references against closed forms."""
import ctypes
import json

import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg
from gemv_dg_bf16_gb300 import _binding as B
from tests import _ref_more as R

A, U = 0x10000, 0x10002                  # fake device addresses: aligned, 2 bytes off
BF, F32, I32, I8 = torch.bfloat16, torch.float32, torch.int32, torch.int8


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_dg_bf16_gb300 import build
    build.build()
    return dg.lib()


def test_i8_argument_errors():
    L = dg.lib()
    call = lambda x=A, q=A, s=A, M=2, K=64: L.dg_quant_i8_rowscale(x, q, s, M, K, None)
    assert call(x=0) == call(q=0) == call(s=0) == call(M=0) == call(K=0) == call(M=-1) == 1
    assert call(K=24) == call(M=2 ** 31 - 255) == call(K=2 ** 31 - 16) == 3
    assert call(x=U) == call(q=U) == call(s=U) == 2
    call = lambda x=A, W=A, s=A, y=A, M=2, N=64, K=256, ws=A, wsb=1 << 30: \
        L.dg_gemv_i8_rowscale(x, W, s, y, M, N, K, ws, wsb, None, None)
    assert call(M=0) == call(M=513) == call(N=0) == call(K=0) == call(x=0) == call(W=0) == call(s=0) == call(y=0) == call(ws=0) == 1
    assert call(K=40) == call(K=131088) == call(N=2 ** 31 - 255) == 3
    assert call(x=U) == call(W=U) == call(s=U) == call(y=U) == call(ws=U) == 2
    need = dg.dg_workspace_bytes(dg.DG_OP_GEMV_I8, 2, 64, 256)
    assert need >= 32768 + 2 * 256 * 2 + 2 * 4 and call(wsb=need - 1) == 4
    assert dg.dg_workspace_bytes(dg.DG_OP_GEMV_I8, 512, 64, 131072) >= 32768 + 512 * 131072 * 2 + 512 * 4


def test_sort_and_rows_argument_errors():
    L = dg.lib()
    call = lambda i=A, o=A, p=A, s=A, M=4, k=2, E=8: L.dg_moe_sort(i, o, p, s, M, k, E, None)
    assert call(i=0) == call(o=0) == call(p=0) == call(s=0) == call(M=0) == call(k=0) == call(E=0) == 1
    assert call(k=33) == call(E=1025) == call(M=2 ** 30, k=2) == 3
    assert call(i=U) == call(o=U) == call(p=U) == call(s=U) == 2
    call = lambda x=A, p=A, o=A, M=4, k=2, P=8, b=64: L.dg_moe_gather(x, p, o, M, k, P, b, None)
    assert call(x=0) == call(p=0) == call(o=0) == call(M=0) == call(k=0) == call(P=0) == call(b=0) == call(b=-16) == 1
    assert call(b=24) == call(k=33) == call(b=2 ** 30 + 16) == 3
    assert call(x=U) == call(p=U) == call(o=U) == 2
    call = lambda z=A, p=A, w=A, y=A, M=4, k=2, P=8, N=64: L.dg_moe_combine(z, p, w or None, y, M, k, P, N, None)
    assert call(z=0) == call(p=0) == call(y=0) == call(M=0) == call(P=0) == call(N=0) == 1
    assert call(N=12) == call(k=40) == 3
    assert call(z=U) == call(p=U) == call(w=U) == call(y=U) == 2
    call = lambda g=A, z=A, p=A, w=A, dz=A, dw=A, M=4, k=2, P=8, N=64: L.dg_moe_combine_grad(g, z, p, w, dz, dw, M, k, P, N, None)
    assert call(g=0) == call(z=0) == call(p=0) == call(w=0) == call(dz=0) == call(dw=0) == call(M=0) == call(k=0) == 1
    assert call(N=4) == call(k=33) == 3
    assert call(g=U) == call(z=U) == call(p=U) == call(w=U) == call(dz=U) == call(dw=U) == 2


def test_logits_argument_errors():
    L = dg.lib()

    def call(x=A, kind=0, ld=100, out=A + 0x100000, ldo=100, M=2, V=100, none=False, **kw):
        e = B.LogitsEdits(**kw)
        return L.dg_logits_adjust(x or None, kind, ld, out or None, ldo, None if none else ctypes.byref(e), M, V, None)
    toks = dict(tokens=A, n_tokens=5, ld_tokens=5)
    assert call(x=0) == call(out=0) == call(M=0) == call(V=0) == call(kind=2) == call(ld=99) == call(ldo=99) == call(none=True) == 1
    assert call(out=A, ldo=101) == 1                              # in place with another stride
    assert call(tokens=A) == call(n_tokens=4) == call(n_tokens=-1, tokens=A) == call(n_bias=3) == call(n_bias=3, bias=A) == call(bias=A, bias_ids=A) == 1
    assert call(lengths=A) == call(prompt_lengths=A) == call(repetition=A) == call(frequency=A) == call(presence=A) == 1
    assert call(**{**toks, "ld_tokens": 4}) == call(mask=A, ld_mask=3) == 1
    assert call(V=2 ** 24 + 1, ld=2 ** 25, ldo=2 ** 25) == call(**{**toks, "n_tokens": 2 ** 24 + 1, "ld_tokens": 2 ** 25}) == 3
    assert call(n_bias=1025, bias=A, bias_ids=A) == 3
    assert call(x=A + 1) == call(x=U, kind=1) == call(out=A + 1) == call(mask=U, ld_mask=4) == call(**{**toks, "tokens": U}) == 2
    assert call(**toks, lengths=U) == call(**toks, repetition=U) == call(n_bias=1, bias=U, bias_ids=A) == call(n_bias=1, bias=A, bias_ids=U) == 2


def test_i8_select_and_table(tmp_path):
    for M, K, v in ((1, 4096, dg.DG_VAR_CC_WARP), (4, 4096, dg.DG_VAR_CC_WARP), (5, 4096, dg.DG_VAR_TC), (512, 4096, dg.DG_VAR_TC),
                    (4, 32768, dg.DG_VAR_CC_WARP), (4, 65536, dg.DG_VAR_TC), (1, 131072, dg.DG_VAR_CC_WARP)):
        assert dg.dg_select(dg.DG_OP_GEMV_I8, M, 4096, K).variant == v, (M, K)

    def check(pick):
        doc = {"format": "libdecodegemm-table",
               "identity": {"arch": "sm_103", "driver": 13000, "runtime": 13000, "build": dg.dg_build_id(),
                            "selection_space": dg.dg_selection_space()},
               "entries": [{"op": "gemv_i8", "M": 4, "N": 64, "K": 64, "pick": pick}]}
        p = tmp_path / "t.json"
        p.write_text(json.dumps(doc))
        return dg.dg_table_check(str(p), "sm_103", 13000, 13000)[0]
    assert check({"variant": 3, "params": [0, 96, 0, 2]}) == 0 and check({"variant": 3, "params": [4, 32, 8, 1]}) == 0
    assert check({"variant": 3, "params": [4, 32, 8]}) == 0 and check({"variant": 1, "params": []}) == 0
    for bad in ({"variant": 1, "params": [4, 8]}, {"variant": 3, "params": [5]}, {"variant": 3, "params": [0, 40]}, {"variant": 3, "params": [0, 144]}, {"variant": 3, "params": [0, 0, 9]},
                {"variant": 3, "params": [0, 0, 0, 3]}, {"variant": 3, "params": [0, 0, 0, 0, 1]}, {"variant": 3, "params": [0, 48, 0, 2]},
                {"variant": 3, "params": [4, 0, 0, 2]}, {"variant": 3, "params": [0, 0, 2, 2]}, {"variant": 3, "params": [-1]}, {"variant": 4, "params": []}):
        assert check(bad) == 6, bad
    assert B._OP_NAMES[dg.DG_OP_GEMV_I8] == "gemv_i8"


def z(shape, t):
    return torch.zeros(shape, dtype=t)


def test_binding_refuses_mismatched_tensors():
    x, pos, w = z((4, 64), BF), z((4, 2), I32), z((4, 2), F32)
    lg = z((2, 64), F32)
    cases = [
        (lambda: dg.dg_quant_i8_rowscale(z((2, 64), F32)), "x: dtype"),
        (lambda: dg.dg_quant_i8_rowscale(x), "x: tensors must be contiguous CUDA"),
        (lambda: dg.dg_gemv_i8_rowscale(z((2, 64), F32), z((8, 64), I8), z((8,), F32)), "x: dtype"),
        (lambda: dg.dg_gemv_i8_rowscale(x, z((8, 64), I8), z((8,), F32)), "x: tensors"),
        (lambda: dg.dg_moe_sort(z((4, 2), torch.int64), 8), "ids: dtype"),
        (lambda: dg.dg_moe_sort(pos, 8), "ids: tensors"),
        (lambda: dg.dg_moe_sort(pos, 2 ** 40, offsets=z((9,), I32)), "a whole number past 32 bits"),
        (lambda: dg.dg_moe_gather(x, pos), "x: tensors"),
        (lambda: dg.dg_moe_combine(z((8, 64), F32), pos), "z: dtype"),
        (lambda: dg.dg_moe_combine(z((8, 64), BF), pos), "z: tensors"),
        (lambda: dg.dg_moe_combine_grad(z((4, 32), BF), z((8, 64), BF), pos, w), "dy: shape"),
        (lambda: dg.dg_logits_adjust(z((2, 8), torch.float16)), "logits: dtype"),
        (lambda: dg.dg_logits_adjust(lg), "logits: rows"),
    ]
    for fn, needle in cases:
        with pytest.raises(ValueError) as e:
            fn()
        assert needle in str(e.value), (needle, str(e.value))


@pytest.mark.parametrize("shape", [(), (64,), (2, 3, 64)])
def test_dimensions(shape):
    x, pos, w = z((4, 64), BF), z((4, 2), I32), z((4, 2), F32)
    cases = [("x", lambda t: dg.dg_quant_i8_rowscale(t(BF))),
             ("x", lambda t: dg.dg_gemv_i8_rowscale(t(BF), z((8, 64), I8), z((8,), F32))),
             ("Wq", lambda t: dg.dg_gemv_i8_rowscale(x, t(I8), z((8,), F32))),
             ("ids", lambda t: dg.dg_moe_sort(t(I32), 8)),
             ("x", lambda t: dg.dg_moe_gather(t(BF), pos)),
             ("pos", lambda t: dg.dg_moe_gather(x, t(I32))),
             ("z", lambda t: dg.dg_moe_combine(t(BF), pos)),
             ("pos", lambda t: dg.dg_moe_combine(x, t(I32))),
             ("z", lambda t: dg.dg_moe_combine_grad(x, t(BF), pos, w)),
             ("logits", lambda t: dg.dg_logits_adjust(t(F32)))]
    for name, call in cases:
        with pytest.raises(ValueError) as e:
            call(lambda dtype: z(shape, dtype))
        assert str(e.value).startswith(f"{name}: shape"), str(e.value)


# ---------------------------------------------------------------- the references themselves

def test_reference_codes_and_linear():
    q, s = R.i8_codes(np.array([[64, 0.25, -3, 1], [0, 0, 0, 0], [np.inf, 1, 0, 0], [256, 4, -12, 1]], np.float32))
    assert q.tolist() == [[127, 0, -6, 2], [0] * 4, [0] * 4, [127, 2, -6, 0]]
    assert abs(s[0] * 127 / 64 - 1) < 2e-7 and s[3] == 4 * s[0] and np.isnan(s[2]) and 0 < s[1] < 1e-30
    y = R.i8_linear(np.array([[64, 1]], np.float32), np.array([[1, -128], [2, 3]], np.int8), np.array([1, 0.5], np.float32))
    s0 = float(s[0])
    assert torch.from_numpy(y).view(BF).tolist() == [[float(torch.tensor((127 - 256) * s0).to(BF)), float(torch.tensor((254 + 6) * s0 * 0.5).to(BF))]]


def test_reference_sort():
    off, pos, slots = R.moe_sort(np.array([[1, 0], [1, 1], [5, -1]], np.int32), 3)
    assert off.tolist() == [0, 1, 3, 3] and pos.tolist() == [[1, 0], [2, -1], [-1, -1]] and slots.tolist() == [1, 0, 2, -1, -1, -1]


def test_reference_edits():
    x = np.array([[1.0, -1.0, 2.0, 3.0, 0.0]], np.float32)
    y = R.adjust(x, tokens=np.array([[0, 1, 2, 2, 9, -1]], np.int32), prompt_lengths=np.array([2]), repetition=np.array([2.0]),
                 frequency=np.array([0.25]), presence=np.array([0.125]), bias_ids=np.array([[3, 3, -1]]), bias=np.array([[1.0, 0.5, 7.0]]),
                 mask=np.array([[0b01111]], np.int32))
    assert y.tolist() == [[0.5, -2.0, 1.0 - 0.5 - 0.125, 4.5, -np.inf]]
