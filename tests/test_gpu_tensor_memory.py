"""Tensor-core kernels of two streams share the SMs: no mix of their CTAs may ask an SM for more tensor memory than it
has, or CTAs of two clusters could wait for each other's.  Shallow rings, which leave room for other CTAs, side by
side, to the bit of what each gives alone."""
import pytest
import torch

import gemv_dg_bf16_gb300 as dg

pytestmark = pytest.mark.gpu

TC = dg.DG_VAR_TC


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _bf(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _i8(M, N, K, *choice):
    g = _gen(M + N)
    x, w = _bf(g, M, K), torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int16).to(torch.int8)
    sw, ws = torch.rand((N,), generator=g, device="cuda"), dg.workspace(dg.DG_OP_GEMV_I8, M, N, K)
    return lambda y: dg.dg_gemv_i8_rowscale(x, w, sw, y=y, ws=ws, choice=dg.Choice.make(TC, *choice)), (M, N), ws


def _bf16(M, N, K, *choice):
    g = _gen(M + N + 1)
    x, w, ws = _bf(g, M, K), _bf(g, N, K), dg.workspace(dg.DG_OP_GEMV_BF16, M, N, K)
    return lambda y: dg.dg_gemv_bf16(x, w, y=y, ws=ws, choice=dg.Choice.make(TC, *choice)), (M, N), ws


def _a8(M, N, K, *choice):
    g = _gen(M + N + 2)
    x, w = _bf(g, M, K), torch.randint(0, 120, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    sw = torch.rand(((N + 127) // 128, (K + 127) // 128), generator=g, device="cuda") * 1e-3
    ws = dg.workspace(dg.DG_OP_GEMV_A8W8, M, N, K)
    return lambda y: dg.dg_gemv_a8w8_blockscale(x, w, sw, y=y, ws=ws, choice=dg.Choice.make(TC, *choice)), (M, N), ws


def _a4(M, N, K, *choice):
    g = _gen(M + N + 3)
    x, ws = _bf(g, M, K), dg.workspace(dg.DG_OP_GEMV_A4W4, M, N, K)
    q, s = dg.dg_quant_fp4_blockscale(_bf(g, N, K), dg.DG_FP4_NV)
    return lambda y: dg.dg_gemv_a4w4_blockscale(x, q, s, dg.DG_FP4_NV, y=y, ws=ws, choice=dg.Choice.make(TC, *choice)), (M, N), ws


CALLS = {"i8 split 16": lambda: _i8(16, 4096, 4096, 2, 16, 8), "i8 split 32": lambda: _i8(32, 4096, 4096, 2, 32, 5),
         "i8 split 48": lambda: _i8(48, 4096, 4096, 2, 48, 3), "i8 pair 64": lambda: _i8(64, 20000, 2048, 0, 64, 0, 2),
         "bf16 split 16": lambda: _bf16(16, 4096, 4096, 2), "bf16 split 128": lambda: _bf16(128, 2048, 4096, 3),
         "a8 64": lambda: _a8(64, 4096, 4096, 2, 1), "a4 128": lambda: _a4(128, 4096, 4096, 2), "a4 16": lambda: _a4(16, 4096, 4096, 2)}


@pytest.mark.parametrize("one,two", [("i8 split 16", "i8 pair 64"), ("i8 split 48", "bf16 split 16"), ("i8 split 16", "a4 16"),
                                     ("i8 split 32", "bf16 split 128"), ("i8 split 32", "a8 64"), ("i8 split 48", "a4 128"),
                                     ("a8 64", "bf16 split 16"), ("a4 128", "a8 64"), ("i8 pair 64", "a4 16"), ("i8 split 16", "i8 split 16")])
def test_two_streams_side_by_side(cuda_device, one, two):
    pair = [CALLS[one](), CALLS[two]()]
    want, got = [], []
    for call, shape, _ in pair:
        y = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        call(y)
        torch.cuda.synchronize()
        want.append(y)
        got.append([torch.full_like(y, 7.0) for _ in range(4)])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for r in range(100):
        for (call, _, _), st, ys in zip(pair, streams, got):
            with torch.cuda.stream(st):
                call(ys[r % 4])
    torch.cuda.synchronize()
    for (_, _, ws), w, ys in zip(pair, want, got):
        for y in ys:
            assert torch.equal(y.view(torch.int16), w.view(torch.int16))
        assert dg.dg_device_status(ws) == 0
