"""The scale of an 8-bit integer row over every finite largest magnitude: how far its code is from 127."""
import numpy as np

F32 = np.float32


def test_largest_magnitudes_reach_127_and_not_128():
    bits = np.arange(0x8000, dtype=np.uint32)                    # every bf16 magnitude
    amax = (bits << 16).view(F32)
    amax = amax[np.isfinite(amax)]
    with np.errstate(under="ignore"):
        A = np.maximum(amax, F32(2.0 ** -100))
        r = F32(127.0) * (F32(1.0) / A)                          # 1 / A may be subnormal
        assert np.isfinite(r).all()
        top = amax * r
    at = top[amax >= F32(2.0 ** -100)].astype(np.float64)
    # r is off by at most 2^-22 (a subnormal 1 / A has 22 bits at least) + 2^-24, the product by 2^-24 more
    assert np.abs(at / 127 - 1).max() <= 2.0 ** -21
    assert np.rint(top).max() == 127 and (np.rint(at) == 127).all()
    assert np.abs(at - 127).max() <= 2.0 ** -14
