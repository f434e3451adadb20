"""The routing's scores to the last bit: without renormalisation the weights are the scores.

Sigmoid: 1 / (1 + exp(-x)), each step rounded to binary32.  Softmax: exp(x - max x) over the exact
sum of these terms rounded to binary32 once.  Two experts that hold all but a trace of a row often
sum to a tie between two floats, which the trace decides.
"""
import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg

pytestmark = pytest.mark.gpu


def _rounded_sum(e):
    """Exact row sums of binary32 values in [0, 1] (whole multiples of 2^-149), rounded to binary32, ties to even."""
    m, x = np.frexp(e)
    whole = np.ldexp(m, 24).astype(np.int64).tolist()
    shift = (x.astype(np.int64) - 24 + 149).tolist()
    out = np.empty(len(e), np.float32)
    for r in range(len(e)):
        s = sum(w << k if k >= 0 else w >> -k for w, k in zip(whole[r], shift[r]))
        drop = max(0, s.bit_length() - 24)
        q, rest = s >> drop, s & ((1 << drop) - 1)
        q += 2 * rest > 1 << drop or (2 * rest == 1 << drop and drop and q & 1)
        out[r] = np.ldexp(np.float64(q), drop - 149)
    return out[:, None]


@pytest.mark.parametrize("E", [8, 32])
@pytest.mark.parametrize("spread", [1.5, 40.0])
def test_scores_bit_for_bit(cuda_device, E, spread):
    """Sigmoid on both sides of -86, where the reciprocal changes its path, softmax terms on both sides of 2^-90."""
    gen = torch.Generator("cuda").manual_seed(E)
    x = spread * torch.randn((20000, E), generator=gen, device="cuda")
    x[::7, 0] = -86.0 + torch.arange(len(x[::7]), device="cuda") % 9 / 4 - 1.0
    for score in (dg.DG_SCORE_SIGMOID, dg.DG_SCORE_SOFTMAX):
        ids, w = dg.dg_moe_route(x, E, score=score, renorm=False)
        if score == dg.DG_SCORE_SIGMOID:
            t = (1.0 + torch.exp(-x)).cpu().numpy()
            p = np.float32(1) / t
        else:
            e = torch.exp(x - x.amax(-1, keepdim=True)).cpu().numpy()
            p = e / _rounded_sum(e)
        assert p.dtype == np.float32
        order = np.argsort(-p.astype(np.float64), axis=-1, kind="stable")
        assert np.array_equal(ids.cpu().numpy(), order)
        want = np.take_along_axis(p, order, -1)
        bad = w.cpu().numpy().view(np.int32) != want.view(np.int32)
        assert not bad.any(), (int(bad.sum()), w.cpu().numpy()[bad][:4], want[bad][:4])
