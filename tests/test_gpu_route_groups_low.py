"""Routing with biases at the type's lowest value over whole runs of experts.

Two such keys sum past binary32's range; the run still holds keys, so it ranks below every run
with larger ones and above a run without any, equal runs by the index.
"""
import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg
from tests import _ref64 as R

pytestmark = pytest.mark.gpu

LOW = float(np.finfo(np.float32).min)


# (experts, runs): runs of a power of two lanes, and runs that are not
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,n_group", [(16, 8), (64, 8), (256, 8), (24, 8), (48, 8), (384, 8), (1024, 8)])
def test_route_lowest_bias_over_whole_runs(cuda_device, E, n_group, sigmoid):
    size, topk_group = E // n_group, 4
    topk = min(32, topk_group * size)
    x = (torch.randint(0, 9, (6, E), generator=torch.Generator().manual_seed(E)).float() / 4).cuda()
    x[1, :size] = -float("inf")                                # a run without any key
    x[2, :] = 0.5
    for first, last in ((2, 6), (0, 4), (0, n_group - 1), (3, n_group - 1)):
        bias = torch.zeros(E, device="cuda")
        bias[first * size:(last + 1) * size] = LOW
        for group_top in (1, 2):
            kw = dict(n_group=n_group, topk_group=topk_group, group_top=group_top)
            ids, w = dg.dg_moe_route(x, topk, score=dg.DG_SCORE_SIGMOID if sigmoid else dg.DG_SCORE_SOFTMAX, bias=bias, **kw)
            ri, rw, _ = R.route(x.cpu().numpy(), topk, sigmoid, bias=bias.cpu().numpy(), **kw)
            # which experts, whatever the order of scores that are a rounding apart
            assert np.array_equal(np.sort(ids.cpu().numpy(), -1), np.sort(ri, -1)), (first, last, group_top)
            assert np.allclose(np.sort(w.cpu().numpy(), -1), np.sort(rw, -1), rtol=1e-5, atol=1e-9)
