"""A shape table's pick for the 8-bit integer linear serves every row count of its bucket: neither depth nor
the width of a group nor the tokens that the CUDA cores take is a condition of a call."""
import json

import pytest
import torch

import gemv_dg_bf16_gb300 as dg

pytestmark = pytest.mark.gpu

CC, TC = dg.DG_VAR_CC_WARP, dg.DG_VAR_TC


@pytest.fixture(scope="module")
def swept(tmp_path_factory, cuda_device):
    """A table of this build and device, to be given other entries."""
    path = tmp_path_factory.mktemp("tab") / "table.json"
    dg.dg_sweep([(dg.DG_OP_GEMV_I8, 1, 64, 64, 0)], str(path), reps=3)
    return json.loads(path.read_text())


def _inputs(M, N, K):
    g = torch.Generator("cuda").manual_seed(N + K + M)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int16).to(torch.int8)
    return x, w, torch.rand((N,), generator=g, device="cuda") * 1e-2 + 1e-4


# A pick's stages fit with the groups and ranks of some rows of the bucket and not with those of others.
@pytest.mark.parametrize("N,K,bucket,first", [(4096, 4096, 128, 97), (4096, 4096, 256, 193), (4099, 12288, 128, 97), (2048, 8192, 96, 65),
                                              (1536, 7168, 384, 257), (24576, 4096, 512, 385), (300, 1040, 16, 13), (300, 1040, 6, 5),
                                              (20480, 5120, 48, 33)])
@pytest.mark.parametrize("variant,params", [(TC, [2]), (TC, [4]), (TC, [6]), (TC, [8]), (TC, [8, 128]), (TC, [8, 128, 4]), (TC, [6, 96, 8]), (TC, [8, 16]),
                                            (TC, [0, 64, 0, 2]), (TC, [0, 96, 0, 2]), (TC, [6, 128, 1, 2]), (CC, [])])
def test_table_pick_serves_every_row_count(cuda_device, swept, tmp_path, N, K, bucket, first, variant, params):
    doc = dict(swept)
    doc["entries"] = [{**swept["entries"][0], "op": "gemv_i8", "M": bucket, "N": N, "K": K,
                       "pick": {"variant": variant, "params": params}}]
    path = tmp_path / "table.json"
    path.write_text(json.dumps(doc))
    rows = range(first, bucket + 1) if N * K < 1 << 24 or bucket <= 64 else sorted({first, first + 1, (first + bucket) // 2, bucket - 16, bucket - 15, bucket})
    x, w, sw = _inputs(bucket, N, K)
    ws = dg.workspace(dg.DG_OP_GEMV_I8, bucket, N, K)
    want = dg.dg_gemv_i8_rowscale(x, w, sw, ws=ws)
    dg.dg_table_load(str(path))
    try:
        for M in rows:
            assert dg.dg_select(dg.DG_OP_GEMV_I8, M, N, K).from_table == 1
            y = dg.dg_gemv_i8_rowscale(x[:M], w, sw, ws=ws)
            assert torch.equal(y.view(torch.int16), want[:M].view(torch.int16)), M
    finally:
        dg.dg_table_clear()
    assert dg.dg_device_status(ws) == 0


def test_explicit_depth_that_does_not_fit_is_refused(cuda_device):
    """A choice given with the call is used as given: eight stages have no room beside 128 tokens."""
    x, w, sw = _inputs(128, 256, 1024)
    for choice in ((TC, 8, 128), (TC, 6, 128, 2), (TC, 4, 128, 4)):
        with pytest.raises(dg.DGError) as e:
            dg.dg_gemv_i8_rowscale(x, w, sw, choice=dg.Choice.make(*choice))
        assert e.value.status == dg.DG_ERR_BAD_VARIANT, choice


@pytest.mark.parametrize("M", [1, 40, 65, 97])
def test_a_pair_takes_groups_that_the_rows_do_not_fill(cuda_device, M):
    N, K = 700, 2064
    x, w, sw = _inputs(M, N, K)
    want = dg.dg_gemv_i8_rowscale(x, w, sw)
    for tokens in (64, 96, 128):
        y = dg.dg_gemv_i8_rowscale(x, w, sw, choice=dg.Choice.make(TC, 0, tokens, 0, 2))
        assert torch.equal(y.view(torch.int16), want.view(torch.int16)), tokens


def test_batch_invariant_mode_takes_table_picks_of_either_family(cuda_device, swept, tmp_path):
    """Every family gives the same bits, so the mode keeps a pick of the CUDA cores, and rows keep theirs in any batch."""
    N, K = 300, 1040
    x, w, sw = _inputs(20, N, K)
    dg.dg_set_numerics(dg.DG_NUMERICS_BATCH_INVARIANT)
    try:
        full = dg.dg_gemv_i8_rowscale(x, w, sw)
        for M in (1, 2, 3, 4, 5):
            assert torch.equal(dg.dg_gemv_i8_rowscale(x[:M], w, sw).view(torch.int16), full[:M].view(torch.int16)), M
        for variant in (CC, TC):
            doc = dict(swept)
            doc["entries"] = [{**swept["entries"][0], "op": "gemv_i8", "M": M, "N": N, "K": K, "pick": {"variant": variant, "params": []}}
                              for M in (3, 4)]                   # (each a bucket of its own)
            path = tmp_path / "table.json"
            path.write_text(json.dumps(doc))
            dg.dg_table_load(str(path))
            for M in (3, 4):
                pick = dg.dg_select(dg.DG_OP_GEMV_I8, M, N, K)
                assert (pick.from_table, pick.variant) == (1, variant)
                assert torch.equal(dg.dg_gemv_i8_rowscale(x[:M], w, sw).view(torch.int16), full[:M].view(torch.int16))
    finally:
        dg.dg_table_clear()
        dg.dg_set_numerics(dg.DG_NUMERICS_FASTEST)
