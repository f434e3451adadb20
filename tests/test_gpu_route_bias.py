"""Biases of any size: key = p + bias in binary32, whatever the bias."""
import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [16, 64, 256, 600])
@pytest.mark.parametrize("n_group", [1, 4])
def test_route_large_and_missing_biases(cuda_device, E, n_group):
    """Biases past 3e38 keep their order, +inf counts as the largest value (equal ones by the index), -inf and NaN leave an expert without a key."""
    if E % n_group:
        pytest.skip("runs of equal size")
    inf, nan = float("inf"), float("nan")
    bias = torch.zeros(E)
    order = {11: inf, 13: inf, 4: 3.4e38, 9: 3.3e38, 2: 3.2e38, 14: 3.05e38, 6: 2.9e38, 1: 1.0e38}
    for e, b in order.items():
        bias[e] = b
    bias[[0, 5]] = -inf
    bias[[3, 7]] = nan
    bias[15] = inf                                             # an expert that is not available all the same
    x = torch.zeros((3, E))
    x[:, 15] = -inf
    for sigmoid in (False, True):
        ids, w = dg.dg_moe_route(x.cuda(), 8, score=dg.DG_SCORE_SIGMOID if sigmoid else dg.DG_SCORE_SOFTMAX, bias=bias.cuda(),
                                 n_group=n_group, topk_group=n_group, renorm=False)
        assert ids.cpu().tolist() == [list(order)] * 3
        want = np.float32(0.5) if sigmoid else np.float32(1.0) / np.float32(E - 1)
        assert (w.cpu().numpy() == want).all()
    if n_group == 1:                                           # experts without a key are never picked
        kw = dict(score=dg.DG_SCORE_SIGMOID, bias=bias[:16].contiguous().cuda())
        ids, _ = dg.dg_moe_route(x[:, :16].contiguous().cuda(), 16, **kw)
        assert ids[0].tolist() == list(order) + [8, 10, 12] + [-1] * 5
