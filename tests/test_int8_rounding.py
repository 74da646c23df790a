"""How far INT8 codes lie from their values: (1/2 + 2^-16) of the scale, as pd.h says of
the append and of each growth of a page's scale. Half a scale alone does not hold: the
reciprocal (or the ratio of scales) and the product with it are each off by up to 2^-24
of themselves, and codes reach 127."""
import numpy as np

from tests import int8_refs as R

MORE = 2.0 ** -16
assert 127 * (2 * 2.0 ** -24 + 2.0 ** -48) < MORE


def off(x, codes, scale):
    """In scales."""
    return np.abs(x.astype(np.float64) / np.float64(scale) - codes).max()


def test_append():
    rng = np.random.default_rng(0)
    worst = 0.0
    for _ in range(20):
        scale = np.float32(2.0 ** rng.uniform(-1, 1))
        x = ((rng.integers(100, 127, 200000) + 0.5) * np.float64(scale)).astype(np.float32)
        x = np.concatenate([x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(1e9))])
        worst = max(worst, off(x, R.quantise(x, np.float32(1) / scale), scale))
    assert 0.5 < worst <= 0.5 + MORE


def test_growth():
    rng = np.random.default_rng(0)
    codes = np.arange(-127, 128, dtype=np.int8)
    worst = 0.0
    for _ in range(2000):
        old, new = np.float32(2.0 ** rng.uniform(-3, 0)), np.float32(2.0 ** rng.uniform(0, 1))
        got = R.quantise(codes, old / new)
        worst = max(worst, off(codes.astype(np.float64) * np.float64(old), got, new))
    assert worst <= 0.5 + MORE
