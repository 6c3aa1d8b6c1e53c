"""The oracle's fused multiply-add of the int8 state update against rational arithmetic, at the sums where a rounding to fp64
on the way would show: products half way between two fp32 values, and addends far below."""
from fractions import Fraction

import numpy as np

import oracle.w8a8 as ow


def nearest32(v):
    """fl32 of a rational number, ties to even."""
    f = np.float32(float(v))
    best = min((np.nextafter(f, np.float32(-np.inf)), f, np.nextafter(f, np.float32(np.inf))),
               key=lambda g: (abs(Fraction(float(g)) - v), int(g.view(np.uint32)) & 1))
    return best


def test_state_update_rounds_once():
    r = np.random.default_rng(11)
    n = 4000
    q = r.integers(-128, 128, n).astype(np.int8)
    q[::2] = r.choice([3, 5, 6, 7, 9, 11, 13, -3, -5, -7], (n + 1) // 2)
    s = (r.integers(2 ** 23, 2 ** 24, n) * 2.0 ** r.integers(-40, 40, n)).astype(np.float32)
    x = (r.choice([-1, 1], n) * r.uniform(1, 2, n) * 2.0 ** r.integers(-90, 20, n)).astype(np.float32)
    one = np.ones((1, 1), np.float32)
    # n rows of one value: delta 0 keeps dA at 1, and then the input's part would be 0, so A is 0 instead
    y, _, _, h = ow.state_update(q.reshape(1, 1, n, 1), s.reshape(1, 1, n), x.reshape(1, 1, n), one.reshape(1, 1, 1), one.reshape(1, 1, 1),
                                 one, np.zeros(1, np.float32))
    want = [nearest32(Fraction(float(a)) * int(b) + Fraction(float(c))) for a, b, c in zip(s, q, x)]
    assert np.array_equal(h.reshape(-1), np.float32(want))
    twice = (s.astype(np.float64) * q + x.astype(np.float64)).astype(np.float32)
    assert (twice != np.float32(want)).sum() > 5, "the inputs reach no sum that rounds differently"
    assert np.array_equal(y.reshape(-1), h.reshape(-1).astype(np.float64))


def test_fma_of_values_that_are_not_finite():
    f = np.float32
    a, b, c = f([np.inf, np.nan, 2.0 ** 100, 2.0 ** 100, 0, 1e-45, -0.0]), f([2, 1, 100, -100, 5, 1, 1]), f([-np.inf, 1, 3e38, 1, -0.0, 1e-45, -0.0])
    want = f([np.nan, np.nan, 3e38 + 100 * 2.0 ** 100, -100 * 2.0 ** 100, 0, 2 * 2.0 ** -149, -0.0])
    assert np.array_equal(ow.fma32(a, b, c), want, equal_nan=True)
    assert np.isinf(ow.fma32(f([2.0 ** 127]), f([100]), f([0])))[0]
