"""The bulk-staged CUDA-core variant fills a stage again only behind its readers: shallow rings, many calls, the bits of
the register-streamed variant."""
import pytest
import torch

import gemv_dg_bf16_gb300 as dg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,stages", [(1, 4096, 4096, 2), (2, 12288, 4096, 2), (4, 4096, 4096, 2), (3, 2048, 1096, 3), (1, 4096, 4096, 0)])
def test_stages_are_filled_behind_their_readers(cuda_device, M, N, K, stages):
    g = torch.Generator("cuda").manual_seed(M + N + K)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn((N, K), generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
    ws = dg.workspace(dg.DG_OP_GEMV_BF16, M, N, K)
    want = dg.dg_gemv_bf16(x, W, ws=ws, choice=dg.Choice.make(dg.DG_VAR_CC_WARP, 4, 8))
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    y = torch.empty_like(want)
    for cps in (1, 2):
        for _ in range(400):
            y.fill_(7.0)
            dg.dg_gemv_bf16(x, W, y=y, ws=ws, choice=dg.Choice.make(dg.DG_VAR_CC_BULK, 0, stages, cps))
            wrong += (y.view(torch.int16) != want.view(torch.int16)).sum()
    assert int(wrong) == 0
    assert dg.dg_device_status(ws) == 0
