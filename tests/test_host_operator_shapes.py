"""Tensors of the wrong number of dimensions are refused with a ValueError that names them, whether
or not the call makes its own buffers (CPU)."""
import pytest
import torch

import gemv_dg_bf16_gb300 as dg

BF, U8, F32 = torch.bfloat16, torch.uint8, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_dg_bf16_gb300 import build
    build.build()
    return dg.lib()


def z(shape, t):
    return torch.zeros(shape, dtype=t)


@pytest.mark.parametrize("shape", [(), (64,), (2, 3, 64)])
def test_dimensions(shape):
    w, s = z((8, 32), U8), z(dg.fp4_scale_shape(8, 64, dg.DG_FP4_NV), U8)
    x = z((2, 64), BF)
    cases = [("x", lambda t: dg.dg_quant_fp4_blockscale(t(BF), dg.DG_FP4_NV)),
             ("q", lambda t: dg.dg_dequant_fp4_blockscale(t(U8), s, dg.DG_FP4_NV)),
             ("x", lambda t: dg.dg_gemv_a4w4_blockscale(t(BF), w, s, dg.DG_FP4_NV)),
             ("Wq", lambda t: dg.dg_gemv_a4w4_blockscale(x, t(U8), s, dg.DG_FP4_NV)),
             ("logits", lambda t: dg.dg_moe_route(t(F32), 2)),
             ("logits", lambda t: dg.dg_logprobs(t(F32)))]
    for name, call in cases:
        with pytest.raises(ValueError) as e:
            call(lambda dtype: z(shape, dtype))
        assert str(e.value).startswith(f"{name}: shape"), str(e.value)
