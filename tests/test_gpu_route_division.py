"""The routing's reciprocals and quotients against IEEE division on the host, to the last bit."""
import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg

pytestmark = pytest.mark.gpu


def _same(got, want):
    assert want.dtype == np.float32
    got = got.cpu().numpy()
    bad = got.view(np.int32) != want.view(np.int32)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("exponent", [-60, -31, -5, -1, 0, 1, 2, 3, 6, 10, 23, 73, 113, 124])
def test_reciprocal_of_every_mantissa(cuda_device, exponent):
    y = (np.arange(1 << 23, dtype=np.uint32) | np.uint32(127 + exponent << 23)).view(np.float32)
    rng = np.random.default_rng(exponent + 100)
    # quotients of at most 1, e not below 2^-90
    e = np.maximum((y * rng.random(y.shape, np.float32)).astype(np.float32), np.float32(2.0 ** -90))
    r, q = dg.dg_selftest_route_division(torch.from_numpy(e).cuda(), torch.from_numpy(y).cuda())
    _same(r, np.float32(1) / y)
    _same(q, e / y)


@pytest.mark.parametrize("seed", range(4))
def test_quotients(cuda_device, seed):
    """Terms from 2^-90 up and sums of both uses; quotients next to a tie among them, and zeros."""
    rng = np.random.default_rng(seed)
    n = 1 << 22
    y = np.exp2(rng.uniform(*((0, 10) if seed % 2 else (-60, 5)), n)).astype(np.float32)
    e = np.exp2(rng.uniform(-90, 0, n)).astype(np.float32)
    half = n // 2                                              # y times a value halfway between two floats
    q = rng.random(half, np.float32) + np.float32(1.0)
    e[:half] = (y[:half].astype(np.float64) * (q.astype(np.float64) + 2.0 ** -24) / 4).astype(np.float32)
    e[::97] = 0.0
    e = np.where((e > 0) & (e < np.float32(2.0 ** -90)), np.float32(2.0 ** -90), e)
    ok = e.astype(np.float64) / y <= 2.0 ** 60
    e = np.where(ok, e, y)
    r, got = dg.dg_selftest_route_division(torch.from_numpy(e).cuda(), torch.from_numpy(y).cuda())
    _same(r, np.float32(1) / y)
    _same(got, e / y)


def test_route_division_refusals(cuda_device):
    a = torch.ones(4, device="cuda")
    with pytest.raises(ValueError):
        dg.dg_selftest_route_division(a, a[:2])
    with pytest.raises(ValueError):
        dg.dg_selftest_route_division(a, a.double())
    L = dg.lib()
    p = a.data_ptr()
    assert L.dg_selftest_route_division(p, p, p, None, 4, None) == dg.DG_ERR_INVALID_ARG
    assert L.dg_selftest_route_division(p, p, p, p, 0, None) == dg.DG_ERR_INVALID_ARG
    assert L.dg_selftest_route_division(p, p + 2, p, p, 1, None) == dg.DG_ERR_ALIGNMENT
