"""Log-probabilities of the longest rows: sums of many equal addends.

A thread folds its running sums away every 256 terms, and those folds are few, so the bound of
short rows holds at every length: (256 + some 200) 2^-24 = 2.8e-5 for the sums and ex2's 2^-22,
4e-5 on a log-probability, 2^-21 of it for its own roundings; the entropy 1e-4 (1 + H).  Equal
addends are the worst case, as every sum between two powers of two rounds the same way.  The
reference is the closed form of a row of two values; the larger one is in every thread's share.
"""
import math

import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg

pytestmark = pytest.mark.gpu


def _closed_form(V, L, d):
    """log-probability of one of the L larger logits, of another, d below, and the entropy."""
    z = L + (V - L) * math.exp(-d)
    return -math.log(z), -d - math.log(z), math.log(z) + d * (V - L) * math.exp(-d) / z


# one row over a cluster of CTAs, and rows enough for one CTA each
@pytest.mark.parametrize("M,V", [(1, 1 << 24), (4, (1 << 24) - 5), (160, 4000037), (160, (1 << 24) - 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [0.0, -float(1 << 22)])     # (sums against the row's largest logit)
def test_logprobs_of_long_rows_of_two_values(cuda_device, M, V, dtype, offset):
    if offset and dtype == torch.bfloat16:
        pytest.skip("no room for differences there")
    if offset:
        M = min(M, 20)
    i = torch.arange(V, device="cuda")
    large = (i % (1 << 20) < 8192) & (i % 4 == 0)
    L = int(large.sum())
    d = 0.5 + torch.arange(M) / 64.0                            # exact in both types
    x = torch.empty((M, V), dtype=dtype, device="cuda")
    x[:] = (offset - d).to(dtype).cuda()[:, None]
    for m in range(M):
        x[m, large] = offset
    d = (x[:, 0].double() - x[:, 1].double()).cpu().numpy()
    tok = torch.zeros(M, dtype=torch.int64, device="cuda")
    r = dg.dg_logprobs(x, tok, n_top=1)
    other = dg.dg_logprobs(x, tok + V - 2)
    ref = np.array([_closed_form(V, L, v) for v in d])
    assert not large[V - 2] and (r["top_ids"] == 0).all()
    assert (r["rank"] == 0).all() and (other["rank"] == L).all()
    for got, want in ((r["logprob"], ref[:, 0]), (r["top_logprobs"][:, 0], ref[:, 0]), (other["logprob"], ref[:, 1])):
        err = np.abs(got.cpu().double().numpy() - want)
        assert (err <= 4e-5 + 2.0 ** -21 * np.abs(want)).all(), err.max()
    err = np.abs(r["entropy"].cpu().double().numpy() - ref[:, 2])
    assert (err <= 1e-4 * (1 + ref[:, 2])).all(), err.max()
