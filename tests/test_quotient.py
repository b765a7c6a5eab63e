"""The encoders' quotient: x r corrected once by its remainder, r = 1 / d rounded, is x / d rounded to nearest.

Away from subnormals and overflow all of its steps scale with powers of two, so that the significands decide: 2^23 of x,
eight of an E4M3 divisor (that of 6 among them). They are gone through here; float64 holds the products exactly."""

import numpy as np
import pytest


@pytest.mark.parametrize("d", [1.0, 1.125, 1.25, 1.375, 1.5, 1.625, 1.75, 1.875])
def test_corrected_quotient_of_every_significand(d):
    x = np.arange(1 << 23, 1 << 24, dtype=np.uint32).astype(np.float32) * np.float32(2.0 ** -23)  # 1 .. 2
    d32 = np.float32(d)
    r = np.float32(1) / d32
    q = x * r
    q64, x64 = q.astype(np.float64), x.astype(np.float64)
    left = q64 * d - x64                       # (28 bits and 24: exact)
    assert np.array_equal(left.astype(np.float32).astype(np.float64), left)  # one fma leaves it exact
    step = left * np.float64(r)                # (48 bits at most: exact)
    s = q64 - step
    got = s.astype(np.float32)
    # s is rounded to 53 bits and then to 24, the fma once: the same unless s lies within 2^-52 of the middle of two fp32
    # values, of which it has to be the exact one
    ulp = np.spacing(np.abs(got)).astype(np.float64)
    middle = np.abs(np.abs(s - got.astype(np.float64)) - ulp / 2) < 2.0 ** -50
    assert not np.any(middle & (step != 0))
    assert np.array_equal(got, x / d32)        # (numpy's division is rounded to nearest)
