"""Negative zeros: code = e2m1(x / (s g)) keeps the sign of a zero quotient."""
import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg
from tests import _ref64 as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [dg.DG_FP4_MX, dg.DG_FP4_NV])
@pytest.mark.parametrize("g", [None, 117.5 / 2688, 3.7e-5])
def test_quant_signs_of_zeros_and_of_what_rounds_to_zero(cuda_device, fmt, g):
    if fmt == dg.DG_FP4_MX and g is not None:
        pytest.skip("MX has no tensor scale")
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((40, 256), generator=gen)
    x[torch.rand(x.shape, generator=gen) < 0.2] = -0.0
    x[torch.rand(x.shape, generator=gen) < 0.2] = 0.0
    x[torch.rand(x.shape, generator=gen) < 0.2] *= 2.0 ** -60      # quotients that round to zero
    x[torch.rand(x.shape, generator=gen) < 0.1] *= 2.0 ** -126     # subnormal ones
    x[3] = -0.0                                                    # blocks of nothing else: zero codes
    x[4] *= 2.0 ** 100
    x[5, 1:] = torch.copysign(torch.zeros(255), x[5, 1:])
    x = x.to(torch.bfloat16).cuda()
    q, s = dg.dg_quant_fp4_blockscale(x, fmt, g=None if g is None else torch.tensor([g], device="cuda"))
    code, byte = R.fp4_quant(x.float().cpu().numpy(), fmt, 1.0 if g is None else g)
    assert (code == 8).any() and np.array_equal(s.cpu().numpy(), R.tile(byte))
    assert np.array_equal(R.unpack(q.cpu().numpy()), code)
