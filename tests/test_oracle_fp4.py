"""Pins of the 4-bit row format's oracle (CPU): every code, ties, ranges, and how far a value may move."""
import numpy as np
import pytest

from oracle import fp4
from oracle.fp8 import e4m3_decode


def test_codes():
    assert fp4.e2m1_decode(range(8)).tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert (fp4.e2m1_encode(fp4.e2m1_decode(range(16))) == np.arange(16)).all()
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert fp4.e2m1_encode(ties).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert (fp4.e2m1_encode(-ties * (1 + 2.0 ** -20)) == 8 + np.arange(1, 8)).all()
    assert fp4.e2m1_encode(np.array([1e9, -7.0])).tolist() == [7, 15]


@pytest.mark.parametrize("power", [0, 30, -30, 119, -133])
def test_rows(power):
    rng = np.random.default_rng(0)
    x = (rng.integers(-255, 256, (40, 64)) * 2.0 ** rng.integers(-9, 1, (40, 64))) * 2.0 ** power
    x[3] = 0
    codes, scales = fp4.quantize_rows(x)
    assert codes.shape == (40, 32) and scales.shape == (40, 8)
    s = np.ascontiguousarray(scales[:, :4]).view(np.float32)[:, 0].astype(np.float64)
    assert (np.frexp(s)[0] == 0.5).all() and s[3] == 1
    amax = np.abs(x).max(-1)
    assert (amax <= 2688 * s).all()
    assert ((amax > 1344 * s) | (amax == 0) | (s == 2.0 ** -126)).all()
    y = fp4.dequantize_rows(codes, scales)
    assert np.isfinite(y).all() and (y[3] == 0).all()
    # half the widest step of a code is t s, and t's rounding (2^-4 of it) may cut 6 t s short of the
    # largest value by 6 * 2^-4 / (1 + 2^-4) < 0.36 t s; blocks under the least scale: 1/4 of a step
    step = (e4m3_decode(scales[:, 4:]) * s[:, None]).repeat(16, -1)
    assert (np.abs(y - x) <= step * (1 + 1e-12)).all()


def test_not_finite():
    """A block's largest value comes back as 6 t s, with t within 2^-4 of a sixth of it."""
    x = np.ones((2, 64))
    x[0, 17], x[1, 40], x[1, 0] = np.inf, np.nan, 4096.0
    y = fp4.dequantize_rows(*fp4.quantize_rows(x))
    assert np.isnan(y[0, 16:32]).all() and (np.abs(np.delete(y[0], range(16, 32)) - 1) <= 2.0 ** -4).all()
    assert np.isnan(y[1, 32:48]).all() and abs(y[1, 0] - 4096.0) <= 256
