"""Sizes of the 4-bit calls next to 2^31: counted in 64 bits, or refused before any launch (CPU)."""
import pytest

import gemv_dg_bf16_gb300 as dg

A = 0x10000                              # a fake device address
TOP = 2 ** 31 - 1
LONG = TOP // 32 * 32                    # the longest row a 32-bit K can state
MOST = 0x7fffff00                        # the longest one, and the most rows, that the calls take


@pytest.fixture(scope="module", autouse=True)
def built():
    from gemv_dg_bf16_gb300 import build
    build.build()
    return dg.lib()


@pytest.mark.parametrize("fmt,block", [(dg.DG_FP4_MX, 32), (dg.DG_FP4_NV, 16)])
@pytest.mark.parametrize("rows,K", [(1, LONG), (TOP, 32), (MOST, 64), (129, MOST), (1000, LONG - 32)])
def test_scale_bytes_of_the_largest_sizes(fmt, block, rows, K):
    assert dg.dg_fp4_scale_bytes(rows, K, fmt) == -(-rows // 128) * -(-(K // block) // 4) * 512


def test_workspace_of_the_longest_rows():
    for M in (1, 512):
        assert dg.dg_workspace_bytes(dg.DG_OP_GEMV_A4W4, M, 64, MOST) >= M * (MOST // 2) + -(-M // 32) * (MOST // 64) * 512


def test_calls_past_the_largest_sizes_are_refused():
    L = dg.lib()
    shape = dg.DG_ERR_UNSUPPORTED_SHAPE
    for fmt in (dg.DG_FP4_MX, dg.DG_FP4_NV):
        for M, K in ((1, LONG), (1, MOST + 32), (TOP, 32)):
            assert L.dg_quant_fp4_blockscale(A, A, A, None, M, K, fmt, None) == shape
            assert L.dg_dequant_fp4_blockscale(A, A, None, A, M, K, fmt, None) == shape
        for N, K in ((64, LONG), (64, MOST + 32), (TOP, 32), (MOST + 1, 32)):
            assert L.dg_gemv_a4w4_blockscale(A, A, A, None, None, A, 1, N, K, fmt, A, 1 << 62, None, None) == shape
