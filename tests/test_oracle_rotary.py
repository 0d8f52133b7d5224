"""Pins of the rotary oracle (no GPU)."""
import numpy as np
import pytest

from oracle import rotary as R


def test_section_layouts_written_out():
    assert R.axis_of_pairs([4]) == [0, 0, 0, 0]
    assert R.axis_of_pairs([2, 3, 1]) == [0, 0, 1, 1, 1, 2]
    assert R.axis_of_pairs([4, 2, 2], interleaved=True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert R.axis_of_pairs([0, 2, 1], interleaved=True) == [1, 2, 1]
    assert R.axis_of_pairs([0, 3]) == [1, 1, 1]


@pytest.mark.parametrize("adjacent", [False, True])
def test_quarter_turn_and_pass_through(adjacent):
    """Position 1 at frequency pi/2 takes (1, 0) to (0, 1); position 0 and
    elements past the rotated ones stay."""
    x = np.zeros((2, 1, 64))
    x[:, 0, 0] = 1.0
    x[:, 0, 40] = 5.0
    f = np.full(16, np.pi / 2)
    y = R.rotate(x, np.array([0, 1]), f, adjacent=adjacent)
    assert np.array_equal(y[0], x[0])
    second = 1 if adjacent else 16
    assert abs(y[1, 0, 0]) < 1e-15 and abs(y[1, 0, second] - 1) < 1e-15 and y[1, 0, 40] == 5.0


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_lengths_and_relative_positions(adjacent, interleaved):
    """Turning keeps lengths, and the dot product of two turned rows depends
    on the difference of their positions on every axis only."""
    rng = np.random.default_rng(1)
    f = rng.random(32).astype(np.float32)
    how = dict(sections=[12, 10, 10], interleaved=interleaved, adjacent=adjacent)
    q, k = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    a, b, shift = (rng.integers(0, 1000, (3, 1)) for _ in range(3))
    y = R.rotate(q, a, f, **how)
    assert np.isclose(np.sum(y * y), np.sum(q * q), rtol=1e-12)
    dot = np.sum(y * R.rotate(k, b, f, **how))
    moved = np.sum(R.rotate(q, a + shift, f, **how) * R.rotate(k, b + shift, f, **how))
    assert np.isclose(dot, moved, rtol=1e-9, atol=1e-9)


def test_each_axis_turns_its_own_pairs():
    x = np.random.default_rng(2).standard_normal((1, 2, 64))
    f = np.ones(32, np.float32)
    sections = [16, 8, 8]
    for axis, (lo, hi) in enumerate([(0, 16), (16, 24), (24, 32)]):
        pos = np.zeros((3, 1), np.int64)
        pos[axis] = 1
        y = R.rotate(x, pos, f, sections=sections)
        moved = np.any(y != x, axis=(0, 1))
        want = np.zeros(64, bool)
        want[lo:hi] = want[32 + lo:32 + hi] = True
        assert np.array_equal(moved, want)
