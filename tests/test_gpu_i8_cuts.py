"""Cuts of the 8-bit integer linear that a choice or a table may name and no default takes: deep rings without a pair
of CTAs, and groups of 128 tokens with K cut -- the bits of the plain reference, or a refusal."""
import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg
from tests import _ref_more as R

pytestmark = pytest.mark.gpu

# (rows that fill no group, one tile and many, blocks of K that the ranks and the rings do not divide)
SHAPES = [(7, 260, 2064), (40, 384, 3088), (128, 130, 1296), (129, 300, 4112), (150, 20000, 2064), (512, 1000, 1168), (200, 129, 9232)]


def _inputs(M, N, K):
    g = torch.Generator().manual_seed(M + N + K)
    x = (torch.randn((M, K), generator=g) * 2).to(torch.bfloat16)
    x[:, ::89] *= 13.0
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int16).to(torch.int8)
    sw = torch.rand((N,), generator=g) * 1e-2 + 1e-4
    return [t.cuda() for t in (x, w, sw)], R.i8_linear(R.f32(x), w.numpy(), sw.numpy())


def _bits(y):
    return y.cpu().view(torch.int16).numpy()


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_deep_rings(M, N, K):
    args, want = _inputs(M, N, K)
    ws = dg.workspace(dg.DG_OP_GEMV_I8, M, N, K)
    ran = {6: 0, 8: 0}
    for tokens in (0, 16, 32, 48, 64, 80, 96, 112, 128):
        for ranks in (0, 1, 2, 3, 5, 8):
            for stages in (6, 8):
                try:
                    y = dg.dg_gemv_i8_rowscale(*args, ws=ws, choice=dg.Choice.make(dg.DG_VAR_TC, stages, tokens, ranks, 1))
                except dg.DGError as e:
                    # eight stages leave room for 112 tokens, and with K cut for 48; six for all, and for 80
                    assert e.status == dg.DG_ERR_BAD_VARIANT
                    assert (tokens == 0 or tokens > 48) and min(tokens or 128, M) > 48 and not (stages == 6 and ranks == 1), (stages, tokens, ranks)
                    continue
                assert not (stages == 8 and tokens == 128 and M > 112), (stages, tokens, ranks)
                ran[stages] += 1
                np.testing.assert_array_equal(_bits(y), want, err_msg=str((stages, tokens, ranks)))
    assert ran[6] >= 30 and ran[8] >= 18
    assert dg.dg_device_status(ws) == 0


@pytest.mark.parametrize("M,N,K", [s for s in SHAPES if s[0] > 112])
def test_wide_groups_with_k_cut(M, N, K):
    args, want = _inputs(M, N, K)
    ws = dg.workspace(dg.DG_OP_GEMV_I8, M, N, K)
    for ranks in (2, 3, 4, 5, 6, 7, 8):
        for stages in (0, 2):
            for _ in range(2):
                y = dg.dg_gemv_i8_rowscale(*args, ws=ws, choice=dg.Choice.make(dg.DG_VAR_TC, stages, 128, ranks))
                np.testing.assert_array_equal(_bits(y), want, err_msg=str((stages, ranks)))
        with pytest.raises(dg.DGError) as e:
            dg.dg_gemv_i8_rowscale(*args, ws=ws, choice=dg.Choice.make(dg.DG_VAR_TC, 4, 128, ranks))
        assert e.value.status == dg.DG_ERR_BAD_VARIANT
    assert dg.dg_device_status(ws) == 0
