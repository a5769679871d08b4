"""The q4_0 format and the rotation as the tests' plain forms have them, pinned by closed forms (CPU)."""
import numpy as np
import pytest

import _q4


def codes_of(x):
    c, s = _q4.quantise(np.asarray(x, np.float32))
    return np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], -1), s


def test_a_grid_of_steps_is_held_exactly():
    for sign in (1, -1):
        x = sign * 0.25 * np.resize(np.arange(-7, 9), 32).astype(np.float32)  # the largest is +-8 steps
        c, s = codes_of(x)
        assert s == np.float16(-sign * 0.25)
        assert np.array_equal(_q4.values(*_q4.quantise(x)), x)
        assert c[15] == 0  # the largest


def test_the_positive_one_of_two_largest_counts():
    x = np.zeros(32, np.float32)
    x[3], x[20] = -4.0, 4.0
    c, s = codes_of(x)
    assert s == -0.5 and c[20] == 0 and c[3] == 15 and c[0] == 8


def test_zero_tiny_and_large_groups():
    c, s = codes_of(np.zeros(32))
    assert s == 0 and (c == 8).all()
    c, s = codes_of(np.full(32, 1e-30))
    assert s == 0 and (c == 8).all()
    c, s = codes_of(np.full(32, 1e6))
    assert s == -65504 and (c == 0).all()


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_a_group_that_is_not_finite_is_nan_and_its_neighbour_is_not(bad):
    x = np.ones(64, np.float32)
    x[40] = bad
    c, s = codes_of(x)
    assert np.isnan(s[1]) and (c[32:] == 8).all() and np.isfinite(s[0])


def test_error_of_random_rows_is_half_a_step_but_at_the_far_end():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((500, 128)).astype(np.float32)
    c, s = _q4.quantise(x)
    err = np.abs(_q4.values(c, s) - x).reshape(500, 4, 32)
    d = np.abs(s.astype(np.float64))[..., None]
    # 7.5 to 8 steps on the other side stay at 7; fp16 rounds the step by 2^-11, eight steps by 8 of those
    assert (err <= d * (1.0 + 8 * 2.0 ** -11)).all()
    near = np.abs(x.reshape(500, 4, 32)) <= 7 * d
    assert (err[near] <= (d * (0.5 + 8 * 2.0 ** -11) + 0 * err)[near]).all()


def test_rotation_closed_forms():
    x = np.arange(1, 65, dtype=np.float32).reshape(1, 1, 64)
    quarter = np.concatenate((np.zeros((1, 8)), np.ones((1, 8))), -1).astype(np.float32)  # 90 degrees
    y = _q4.rotate(x, quarter, np.array([0]), False)
    assert np.array_equal(y[0, 0, :8], -x[0, 0, 8:16]) and np.array_equal(y[0, 0, 8:16], x[0, 0, :8])
    assert np.array_equal(y[0, 0, 16:], x[0, 0, 16:])
    y = _q4.rotate(x, quarter, np.array([0]), True)
    assert np.array_equal(y[0, 0, 0:16:2], -x[0, 0, 1:16:2]) and np.array_equal(y[0, 0, 1:16:2], x[0, 0, 0:16:2])


def test_rotation_keeps_angles_between_positions():
    rng = np.random.default_rng(1)
    t = _q4.table(200, 64)
    q, k = rng.standard_normal((2, 1, 1, 64)).astype(np.float32)
    for interleaved in (False, True):
        def dot(i, j):
            a, b = (_q4.rotate(x, t, np.array([p]), interleaved).astype(np.float64) for x, p in ((q, i), (k, j)))
            return float((a * b).sum())
        assert abs(dot(150, 140) - dot(10, 0)) < 1e-4 and abs(dot(150, 140) - dot(10, 5)) > 1e-3
