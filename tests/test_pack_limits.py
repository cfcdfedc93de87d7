"""Pins of packed rows at the largest finite numbers, and at the border below
which nothing is special."""
import numpy as np

from oracle import train as R

MAX = float(np.finfo(np.float32).max)
EDGE = float(127 * 2.0 ** 121)


def test_the_largest_numbers_stay_finite():
    x = np.zeros((1, 96))
    x[0, :4] = MAX, -MAX, 2.0 ** 120, 3 * 2.0 ** 120
    x[0, 32], x[0, 33] = EDGE, 2.0 ** 121
    x[0, 64], x[0, 65] = float(np.nextafter(np.float32(EDGE), np.float32(INF))), -2.0 ** 127
    q, s = R.pack(x)
    # 2^121 is the largest step: its 127-fold is a float, twice the step's is not
    assert s.tolist() == [[248, 248, 248]]
    assert q[0, :4].tolist() == [127, -127, 0, 2]
    assert q[0, 32:34].tolist() == [127, 1] and q[0, 64:66].tolist() == [127, -64]
    v = R.unpack(q, s)
    assert np.isfinite(v.astype(np.float32)).all()
    # within a step where the largest is past 127 steps, else within half of one
    assert abs(v[0, 0] - MAX) < 2.0 ** 121 and v[0, 32] == EDGE


INF = float("inf")


def test_no_block_of_floats_needs_more_than_127_steps_below_the_edge():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(40, 64)) * np.exp2(rng.integers(100, 125, size=(40, 1)))
    x = np.clip(x, -EDGE, EDGE)
    q, s = R.pack(x)
    step = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, 1)
    assert s.max() <= 248 and np.all(np.abs(R.unpack(q, s) - x) <= step / 2)
