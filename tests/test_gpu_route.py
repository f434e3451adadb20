"""Routing of tokens to experts against a plain 64-bit reference.

A key's binary32 error is below 1e-6 (a few roundings of values up to about 2), so rows
whose closest decision has a margin above 2e-6 -- true ties aside, which go by the index --
must pick the reference's experts; gate weights agree to 1e-5 relative.
"""
import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg
from tests import _ref64 as R

pytestmark = pytest.mark.gpu


def _check(x, topk, least=0.9, **kw):
    sig = kw.pop("sigmoid")
    bias = kw.get("bias")
    ids, w = dg.dg_moe_route(x, topk, score=dg.DG_SCORE_SIGMOID if sig else dg.DG_SCORE_SOFTMAX, **kw)
    kw["bias"] = None if bias is None else bias.cpu().numpy()
    ri, rw, margin = R.route(x.float().cpu().numpy(), topk, sig, **kw)
    ids, w = ids.cpu().numpy(), w.cpu().double().numpy()
    sure = margin > 2e-6
    assert sure.mean() >= least
    assert np.array_equal(ids[sure], ri[sure])
    assert np.allclose(w[sure], rw[sure], rtol=1e-5, atol=1e-9)
    for r in ids:                                              # every row: distinct experts or -1
        live = r[r >= 0]
        assert len(set(live.tolist())) == len(live) and (live < x.shape[1]).all()
    return ids, w


def _logits(M, E, seed, dtype=torch.float32):
    return (1.5 * torch.randn((M, E), generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


SHAPES = [(1, 1, 1), (3, 2, 2), (5, 31, 4), (2, 32, 32), (16, 33, 6), (16, 64, 8), (7, 96, 5), (9, 128, 6), (4, 160, 6),
          (33, 255, 10), (64, 256, 8), (3, 384, 8), (5, 513, 16), (2, 1000, 20), (3, 1024, 32)]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("M,E,topk", SHAPES)
def test_route_without_groups(cuda_device, M, E, topk, sigmoid, dtype, with_bias):
    bias = 0.1 * torch.randn((E,), generator=torch.Generator().manual_seed(E)).cuda() if with_bias else None
    _check(_logits(M, E, M * E, dtype), topk, sigmoid=sigmoid, bias=bias, renorm=bool(M % 2), scale=2.5, least=0.6)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("M,E,n_group,topk_group,topk", [
    (16, 256, 8, 4, 8), (9, 64, 8, 3, 6), (5, 160, 8, 3, 6), (7, 48, 3, 2, 5), (4, 384, 8, 4, 8), (6, 1024, 16, 14, 32),
    (8, 32, 32, 5, 5), (5, 60, 4, 1, 15), (3, 1000, 8, 2, 9), (4, 96, 2, 1, 7), (6, 512, 32, 3, 12)])
def test_route_groups(cuda_device, M, E, n_group, topk_group, topk, group_top, sigmoid):
    bias = 0.05 * torch.randn((E,), generator=torch.Generator().manual_seed(E)).cuda()
    for b in (None, bias):
        _check(_logits(M, E, M + E), topk, sigmoid=sigmoid, bias=b, n_group=n_group, topk_group=topk_group,
               group_top=group_top, least=0.6)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("n_group", [1, 4])
def test_route_ties_go_to_the_lowest_index(cuda_device, sigmoid, n_group):
    """Logits of a handful of values, and rows of one value: exact ties everywhere."""
    x = torch.randint(-2, 3, (40, 64), generator=torch.Generator().manual_seed(3)).float()
    x[5] = 0.25
    x[6] = -7.0
    ids, _ = _check(x.cuda(), 8, sigmoid=sigmoid, n_group=n_group, topk_group=max(1, n_group // 2), group_top=2, least=1.0)
    assert ids[5].tolist() == list(range(8)) and ids[6].tolist() == list(range(8))


@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_masked_experts_and_odd_values(cuda_device, sigmoid):
    inf, nan = float("inf"), float("nan")
    x = _logits(12, 64, 1)
    x[0] = -inf                                                # nothing available
    x[1, 3:] = -inf                                            # fewer than topk
    x[2, ::2] = nan
    x[3] = nan
    x[4, 7] = inf
    x[5] = -3.0e38                                             # the type's lowest: available, all equal
    x[6, 10:] = -3.4028234663852886e38
    x[7] = 200.0
    x[8] = -200.0                                              # sigmoid underflows to 0: weights 0
    x[9, :32] = -inf                                           # whole runs unavailable
    for kw in (dict(), dict(n_group=4, topk_group=2, group_top=2), dict(n_group=4, topk_group=1, group_top=1)):
        ids, w = _check(x.clone(), 8, sigmoid=sigmoid, least=0.5, **kw)
        assert (ids[0] == -1).all() and (w[0] == 0).all() and (ids[3] == -1).all()
        assert sorted(ids[1][ids[1] >= 0].tolist()) == [0, 1, 2] and (w[1][ids[1] < 0] == 0).all()
        assert 7 == ids[4][0]
        assert np.isfinite(w).all()
        assert ids[5].tolist() == list(range(8))


def test_route_strided_and_misaligned_logits(cuda_device):
    for dtype in (torch.float32, torch.bfloat16):
        base = _logits(20, 200, 5, dtype)
        ref = dg.dg_moe_route(base[:, 3:131].contiguous(), 6, score=dg.DG_SCORE_SIGMOID)
        got = dg.dg_moe_route(base[:, 3:131], 6, score=dg.DG_SCORE_SIGMOID)
        assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_route_a_row_does_not_depend_on_the_batch(cuda_device):
    for E in (64, 200, 256):
        x = _logits(500, E, E)
        b = 0.1 * torch.randn((E,), device="cuda")
        kw = dict(score=dg.DG_SCORE_SOFTMAX, bias=b, n_group=4, topk_group=2, group_top=2)
        ids, w = dg.dg_moe_route(x, 8, **kw)
        for M in (1, 3, 4, 5, 33, 499):
            i2, w2 = dg.dg_moe_route(x[:M].contiguous(), 8, **kw)
            assert torch.equal(i2, ids[:M]) and torch.equal(w2, w[:M])


def test_route_many_rows_and_long_strides(cuda_device):
    """70,000 rows, and a row stride that takes offsets past 2^31 elements."""
    x = _logits(1000, 128, 2)
    ids, w = dg.dg_moe_route(x, 6)
    i2, w2 = dg.dg_moe_route(x.repeat(70, 1), 6)
    assert torch.equal(i2, ids.repeat(70, 1)) and torch.equal(w2, w.repeat(70, 1))
    far = torch.empty((3, 1 << 30), dtype=torch.bfloat16, device="cuda")
    far[:, :128] = x[:3].to(torch.bfloat16)
    a, b = dg.dg_moe_route(far[:, :128], 6), dg.dg_moe_route(x[:3].to(torch.bfloat16), 6)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_route_feeds_the_expert_products(cuda_device):
    """The ids and weights go straight into the MoE calls, a masked slot included."""
    from synth import decode_inputs as S
    W1q, s1, W2q, s2 = S.moe_weights(16, 64, 256, 128, device=cuda_device)
    x, _, _ = S.moe_inputs(4, 256, 6, 16, device=cuda_device)
    logits = _logits(4, 16, 9)
    logits[2, 4:] = -float("inf")                              # 4 experts for 6 slots
    ids, w = dg.dg_moe_route(logits, 6)
    y = dg.dg_moe_w2(dg.dg_moe_w1_silu(x, ids, W1q, s1), ids, w, W2q, s2)
    one = dg.dg_moe_w2(dg.dg_moe_w1_silu(x[2:3].contiguous(), ids[2:3, :4].contiguous(), W1q, s1),
                       ids[2:3, :4].contiguous(), w[2:3, :4].contiguous(), W2q, s2)
    assert torch.isfinite(y).all() and torch.allclose(y[2:3].float(), one.float(), rtol=2e-2, atol=1e-3)


def test_route_refusals(cuda_device):
    x = _logits(2, 64, 1)
    for kw, status in ((dict(topk=0), 1), (dict(topk=33), 3), (dict(topk=8, n_group=3), 3), (dict(topk=8, n_group=0), 1),
                       (dict(topk=9, n_group=8, topk_group=1), 3), (dict(topk=2, n_group=8, topk_group=9), 1),
                       (dict(topk=2, group_top=3), 1), (dict(topk=2, score=2), 1), (dict(topk=2, n_group=64), 3)):
        with pytest.raises(dg.DGError) as e:
            dg.dg_moe_route(x, **kw)
        assert e.value.status == status, kw
    with pytest.raises(dg.DGError):
        dg.dg_moe_route(_logits(1, 1025, 1), 2)
