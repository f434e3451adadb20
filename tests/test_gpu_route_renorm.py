"""Gate weights to the last bit: w = p / sum p correctly rounded, then times scale.

The sum is taken over 32 slots in binary32, pairwise over slot distances 16, 8, 4, 2, 1 (slots past
topk are 0); p comes from the same call without renormalisation.
"""
import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,topk", [(8, 2), (64, 6), (256, 8), (128, 32), (512, 10)])
@pytest.mark.parametrize("scale", [1.0, 2.5])
def test_route_weights_are_correctly_rounded_quotients(cuda_device, E, topk, sigmoid, scale):
    x = (1.5 * torch.randn((4000, E), generator=torch.Generator().manual_seed(E + topk))).cuda()
    x[0] = -80.0                                               # weights that are all but subnormal
    x[1] = -200.0                                              # and ones that underflow
    kw = dict(score=dg.DG_SCORE_SIGMOID if sigmoid else dg.DG_SCORE_SOFTMAX)
    ids, p = dg.dg_moe_route(x, topk, renorm=False, **kw)
    i2, w = dg.dg_moe_route(x, topk, renorm=True, scale=scale, **kw)
    assert torch.equal(ids, i2)
    t = np.zeros((x.shape[0], 32), np.float32)
    t[:, :topk] = p.cpu().numpy()
    for o in (16, 8, 4, 2, 1):
        t = t + t[:, np.arange(32) ^ o]
    p = p.cpu().numpy()
    with np.errstate(divide="ignore", invalid="ignore"):
        want = np.where(t[:, :1] > 0, p / t[:, :1], np.float32(0)) * np.float32(scale)
    assert want.dtype == np.float32
    assert np.array_equal(w.cpu().numpy().view(np.int32), want.view(np.int32))
