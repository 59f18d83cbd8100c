"""The chosen-block oracle against hand-worked cases (no GPU)."""
import numpy as np

from oracle import blocks


def test_bounds_of_a_ragged_run():
    k = np.array([[1.0, -2.0], [3.0, 0.0], [-1.0, 5.0]])
    hi, lo = blocks.bounds(k, 2)
    assert hi.tolist() == [[3.0, 0.0], [-1.0, 5.0]] and lo.tolist() == [[1.0, -2.0], [-1.0, 5.0]]


def test_score_takes_the_better_end_of_each_channel_and_the_best_head():
    hi, lo = np.array([[3.0, 0.0]]), np.array([[1.0, -2.0]])
    assert blocks.scores([[2.0, 1.0]], hi, lo).tolist() == [6.0]
    assert blocks.scores([[2.0, -1.0]], hi, lo).tolist() == [8.0]
    assert blocks.scores([[-1.0, 0.0], [0.0, -3.0]], hi, lo).tolist() == [6.0]


def test_score_bounds_every_key():
    r = np.random.default_rng(0)
    k, q = r.standard_normal((64, 16)), r.standard_normal((3, 16))
    s = blocks.scores(q, *blocks.bounds(k, 16))
    top = (k @ q.T).max(1).reshape(4, 16).max(1)
    assert (s >= top).all()


def test_sums_are_exact():
    hi = np.array([[1e16, 1.0, -1e16], [1.0, 0.0, 0.0]])
    assert blocks.scores([[1.0, 1.0, 1.0]], hi, hi).tolist() == [1.0, 1.0]


def test_choice():
    s = [5.0, 1.0, 7.0, 7.0, 7.0, 0.0]
    assert blocks.choose(s, 2, 0, 0).tolist() == [2, 3]        # ties to the lowest
    assert blocks.choose(s, 3, 1, 1).tolist() == [0, 2, 5]
    assert blocks.choose(s, 2, 1, 1).tolist() == [0, 5]        # nothing left to choose
    assert blocks.choose(s[:2], 4, 1, 1).tolist() == [0, 1, -1, -1]
    assert blocks.choose([], 2, 0, 0).tolist() == [-1, -1]


def test_rows():
    assert blocks.rows_of([0, 2, -1], 3, 8) == [0, 1, 2, 6, 7]
