"""A slot of the weights' ring is filled again only behind its readers: calls whose rings turn over fastest, many
times over, to the bit.  (Slots handed back too early showed in up to one call of a hundred of the first kind.)"""
import pytest
import torch

import gemv_dg_bf16_gb300 as dg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,choice,calls", [(512, 24576, 4096, (6, 128, 1, 1), 600), (512, 24576, 4096, (2, 0, 0, 0), 400),
                                                (448, 24576, 4096, (4, 128, 1, 1), 400), (300, 1536, 7168, (4, 112, 3, 1), 1500),
                                                (336, 1536, 7168, (), 1500), (256, 4096, 4096, (2, 128, 4, 0), 800),
                                                (77, 4099, 12288, (), 600), (16, 4096, 4096, (2, 0, 2, 0), 800), (512, 24576, 4096, (), 400)])
def test_slots_are_filled_behind_their_readers(cuda_device, M, N, K, choice, calls):
    g = torch.Generator("cuda").manual_seed(M + N + K)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int16).to(torch.int8)
    sw = torch.rand((N,), generator=g, device="cuda") * 1e-2 + 1e-4
    q, s = dg.dg_quant_i8_rowscale(x)
    # exact sums (products of 64-bit numbers), then each step rounded to binary32 as the definition has it
    want = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    for n in range(0, N, 4096):
        sums = (q.double() @ w[n:n + 4096].double().t()).to(torch.int32)
        want[:, n:n + 4096] = (sums.float() * (s[:, None] * sw[None, n:n + 4096])).to(torch.bfloat16)
    ws = dg.workspace(dg.DG_OP_GEMV_I8, M, N, K)
    y = torch.empty_like(want)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    pick = dg.Choice.make(dg.DG_VAR_TC, *choice)
    for _ in range(calls):
        y.fill_(7.0)
        dg.dg_gemv_i8_rowscale(x, w, sw, y=y, ws=ws, choice=pick)
        wrong += (y.view(torch.int16) != want.view(torch.int16)).sum()
    assert int(wrong) == 0
    assert dg.dg_device_status(ws) == 0
