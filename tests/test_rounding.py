"""The quantisers' rounding to whole codes, on the CPU: fl(x + c) truncated, with c
the fp32 number below one half carrying x's sign, against half away from zero."""
import numpy as np
import pytest

HALF = np.float32(float.fromhex("0x1.fffffep-2"))


def truncated_sum(x):
    x = np.asarray(x, np.float32)
    return np.trunc(x + np.copysign(HALF, x)).astype(np.int64)


def half_away(x):
    x = np.asarray(x, np.float64)
    return np.copysign(np.floor(np.abs(x) + 0.5), x).astype(np.int64)


def test_the_sum_is_the_rounding_for_every_value_below_256():
    """Both are steps that never fall as x grows (a sum with a constant is
    rounded monotonically, a truncation is monotone), and odd in x: they agree
    on [0, 256) if they agree at 0, at each tie n + 1/2, and at the fp32 numbers
    next to it."""
    tie = np.arange(0, 256, dtype=np.float32) + np.float32(0.5)
    assert np.nextafter(HALF, np.float32(1)) == 0.5
    for x in (np.zeros(1, np.float32), tie, np.nextafter(tie, np.float32(0)), np.nextafter(tie, np.float32(300))):
        x = x[x < 256]
        assert np.array_equal(truncated_sum(x), half_away(x)) and np.array_equal(truncated_sum(-x), half_away(-x))


@pytest.mark.parametrize("top", [7, 127])
def test_no_product_rounds_past_the_largest_code(top):
    """v (1 / d) with d = amax / top, each rounded: at most top (1 + 2^-22), which
    the rounding takes to top."""
    v = np.random.default_rng(top).uniform(1e-30, 1e30, 100000).astype(np.float32)
    t = v * (np.float32(1) / (v / np.float32(top)))
    assert (np.abs(t / np.float64(top) - 1) <= 2.0 ** -22).all() and (truncated_sum(t) == top).all()
