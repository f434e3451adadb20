"""The batch-invariant mode asks nothing of the 8-bit integer linear, whose families give the same bits."""
import pytest

import gemv_dg_bf16_gb300 as dg


@pytest.mark.parametrize("M,K", [(1, 4096), (2, 64), (4, 4096), (4, 32768), (4, 65536), (1, 131072), (5, 4096), (512, 4096)])
def test_batch_invariant_mode_keeps_the_fastest_family(M, K):
    from gemv_dg_bf16_gb300 import build
    build.build()
    fastest = dg.dg_select(dg.DG_OP_GEMV_I8, M, 4096, K)
    dg.dg_set_numerics(dg.DG_NUMERICS_BATCH_INVARIANT)
    try:
        c = dg.dg_select(dg.DG_OP_GEMV_I8, M, 4096, K)
        assert c.as_tuple() == fastest.as_tuple()
        assert dg.dg_select(dg.DG_OP_GEMV_BF16, 1, 4096, 4096).variant == dg.DG_VAR_TC      # (the others change family)
    finally:
        dg.dg_set_numerics(dg.DG_NUMERICS_FASTEST)
