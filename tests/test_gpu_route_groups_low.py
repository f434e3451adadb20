"""Routing with biases at the type's lowest value over whole runs of experts.

Two such keys sum past binary32's range, to -inf; the run still holds keys, so it ranks below every
run with a larger sum and above a run without any key, equal runs by the index.
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


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,n_group", [(32, 8), (256, 8), (24, 8), (384, 8), (1024, 16)])
def test_route_run_with_one_expert_left_ranks_above_runs_with_none(cuda_device, E, n_group, sigmoid):
    """Its two best keys sum to the lowest value, those of a run of lowest keys to less; runs without keys come last."""
    size = E // n_group
    x = (torch.randint(0, 9, (4, E), generator=torch.Generator().manual_seed(E)).float() / 4).cuda()
    x[1, :2 * size] = -float("inf")                            # two runs without keys in front
    bias = torch.full((E,), LOW, device="cuda")
    for live in ((n_group - 1, n_group - 2), (3, 5)):
        b = bias.clone()
        for k in live:
            b[k * size + size // 2] = 0.0
        for topk_group in (1, 2, 4, n_group):
            topk = min(32, topk_group * size)
            kw = dict(n_group=n_group, topk_group=topk_group, group_top=2)
            ids, w = dg.dg_moe_route(x, topk, score=dg.DG_SCORE_SIGMOID if sigmoid else dg.DG_SCORE_SOFTMAX, bias=b, **kw)
            ri, rw, _ = R.route(x.cpu().numpy(), topk, sigmoid, bias=b.cpu().numpy(), **kw)
            assert np.array_equal(np.sort(ids.cpu().numpy(), -1), np.sort(ri, -1)), (live, topk_group)
            assert np.allclose(np.sort(w.cpu().numpy(), -1), np.sort(rw, -1), rtol=1e-5, atol=1e-9)
