"""Logits next to both ends of their type: a log-probability is -inf only where scale (z - max) leaves
binary32's range, not where z - max does.

Bound: the three roundings of scale (z - max) and the sum's, 2^-21 of the value.
"""
import math

import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1.0, 0.7, 0.01, 1e-6, 3.0])
@pytest.mark.parametrize("V", [7, 300, 70001])
def test_logprobs_across_the_whole_range(cuda_device, dtype, scale, V):
    top, low = torch.finfo(dtype).max, torch.finfo(dtype).min
    rows = [(top / 4, low), (top, low), (top, -top / 2), (1.0, low), (0.0, low / 2), (top / 2, low / 2)]
    x = torch.empty((len(rows), V), dtype=dtype)
    for m, (a, b) in enumerate(rows):
        x[m] = b
        x[m, V // 2] = a
    x = x.cuda()
    tok = torch.full((len(rows),), V - 1, device="cuda")
    r = dg.dg_logprobs(x, tok, n_top=2, scale=scale)
    s = float(np.float32(scale))
    z = x.double().cpu().numpy()
    want = s * (z[:, V - 1] - z[:, V // 2])                    # (log of the sum is 0: every other term underflows)
    want = np.where(np.abs(want) > 3.4028235677973366e38, -math.inf, want)
    for got in (r["logprob"], r["top_logprobs"][:, 1]):
        got = got.cpu().double().numpy()
        fin = np.isfinite(want)
        assert np.array_equal(got[~fin], want[~fin])
        assert (np.abs(got[fin] - want[fin]) <= 2.0 ** -21 * np.abs(want[fin])).all(), (got, want)
    assert (r["top_logprobs"][:, 0] == 0).all() and (r["entropy"] == 0).all() and (r["rank"] == 1).all()
    assert (r["top_ids"][:, 0] == V // 2).all() and (r["top_ids"][:, 1] == 0).all()
