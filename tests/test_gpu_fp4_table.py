"""A shape table's pick for the 4-bit linear serves both formats, every row count of its bucket and
both K-split rules: pipeline depth is no condition of a call."""
import json

import pytest
import torch

import gemv_dg_bf16_gb300 as dg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swept(tmp_path_factory, cuda_device):
    """A table of this build and device, to be given other entries."""
    path = tmp_path_factory.mktemp("tab") / "table.json"
    dg.dg_sweep([(dg.DG_OP_GEMV_A4W4, 1, 64, 64, dg.DG_FP4_MX)], str(path), reps=3)
    return json.loads(path.read_text())


@pytest.mark.parametrize("N,K,bucket,rows", [(24576, 4096, 1, (1,)), (8192, 4096, 256, (193, 256)),
                                             (2048, 5120, 384, (257, 300, 320, 384)), (4096, 4096, 64, (49, 64)),
                                             (4096, 12288, 16, (13, 16)), (300, 1056, 4, (4,))])
@pytest.mark.parametrize("stages", [2, 5, 7, 8])
def test_table_pick_serves_formats_row_counts_and_modes(cuda_device, swept, tmp_path, N, K, bucket, rows, stages):
    doc = dict(swept)
    doc["entries"] = [{**swept["entries"][0], "op": "gemv_a4w4", "M": bucket, "N": N, "K": K,
                       "pick": {"variant": dg.DG_VAR_TC, "params": [stages, 0, 0, 0, 0, 0]}}]
    path = tmp_path / "table.json"
    path.write_text(json.dumps(doc))
    gen = torch.Generator("cuda").manual_seed(N + K)
    w = (torch.randn((N, K), generator=gen, device="cuda") * K ** -0.5).to(torch.bfloat16)
    x = torch.randn((max(rows), K), generator=gen, device="cuda").to(torch.bfloat16)
    calls = [(fmt, M, mode) for fmt in (dg.DG_FP4_MX, dg.DG_FP4_NV) for M in rows
             for mode in (dg.DG_NUMERICS_FASTEST, dg.DG_NUMERICS_BATCH_INVARIANT)]
    packed = {fmt: dg.dg_quant_fp4_blockscale(w, fmt) for fmt in (dg.DG_FP4_MX, dg.DG_FP4_NV)}

    def run(fmt, M, mode):
        dg.dg_set_numerics(mode)
        return dg.dg_gemv_a4w4_blockscale(x[:M], *packed[fmt], fmt)
    try:
        want = [run(*c) for c in calls]
        dg.dg_table_load(str(path))
        try:
            for c, y in zip(calls, want):
                assert dg.dg_select(dg.DG_OP_GEMV_A4W4, c[1], N, K).from_table == 1
                assert torch.equal(run(*c).view(torch.int16), y.view(torch.int16)), c
        finally:
            dg.dg_table_clear()
    finally:
        dg.dg_set_numerics(dg.DG_NUMERICS_FASTEST)


def test_explicit_depth_that_does_not_fit_is_refused(cuda_device):
    """A choice given with the call is used as given."""
    N, K, M = 24576, 4096, 1
    w = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    x = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    q, s = dg.dg_quant_fp4_blockscale(w, dg.DG_FP4_NV)
    with pytest.raises(dg.DGError) as e:
        dg.dg_gemv_a4w4_blockscale(x, q, s, dg.DG_FP4_NV, choice=dg.Choice.make(dg.DG_VAR_TC, 8))
    assert e.value.status == dg.DG_ERR_BAD_VARIANT
