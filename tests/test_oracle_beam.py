"""The beam search oracle on examples done by hand (CPU)."""

import math

import numpy as np

from oracle import beam


def test_select_by_hand():
    # p = 1/2, 1/4, 1/4 and 1/8, 7/8 under scores 0 and -1: the ties of row 0 by token
    x = [[[math.log(2), 0.0, 0.0, -math.inf], [0.0, math.log(7), -math.inf, -math.inf]]]
    s, p, t, f = beam.select(x, [[0.0, -1.0]], 6, end_token=2)
    assert p == [[0, 1, 0, 0, 1, -1]] and t == [[0, 1, 1, 2, 0, -1]]
    want = [math.log(0.5), math.log(0.875) - 1, math.log(0.25), math.log(0.25),
            math.log(0.125) - 1, -math.inf]
    np.testing.assert_allclose(s[0], want, rtol=1e-14)
    assert f == [[False, False, False, True, False, False]]
    # a finished beam keeps its score; a dead one has nothing
    s, p, t, f = beam.select([x[0] + x[0]], [[0.0, -0.5, -math.inf, math.nan]], 3,
                             [[False, True, False, False]], 3)
    assert p == [[1, 0, 0]] and t == [[3, 0, 1]] and s[0][0] == -0.5 and f == [[True, False, False]]


def test_reorder_by_hand():
    # two beams share page 5; beam 1 is dropped, beam 0 doubled: its page 6 (2 tokens) is copied
    # onto 7, which beam 1 gave back
    r = beam.reorder([[0, 0]], [18, 18], [[5, 6], [5, 7]], [9], 16, 10)
    assert r["rows"] == [[5, 6], [5, 7]] and r["copies"] == [(-1, -1, 0), (6, 7, 2)]
    assert r["free"] == [9] and r["lens"] == [18, 18]
    # whole pages are shared, not copied
    r = beam.reorder([[1, 1]], [32, 32], [[5, 6], [5, 7]], [9], 16, 10)
    assert r["rows"] == [[5, 7], [5, 7]] and r["free"] == [9, 6]
    assert r["copies"] == [(-1, -1, 0)] * 2
    # the end of a request gives each page back once
    r = beam.reorder([[-1, -1]], [18, 18], [[5, 6], [5, 7]], [9], 16, 10)
    assert r["rows"] == [[], []] and r["free"] == [9, 5, 6, 7] and r["lens"] == [0, 0]
    # no page for the second request's copy: it stays; so does a malformed one
    r = beam.reorder([[0, 3], [0, 0], [1, 0]], [2, 2, 3, 0, 4, 4], [[1], [2], [3], [8], [4], [5]], [],
                     16, 9)
    assert r["bad"] == [0] and r["fail"] == 1 and r["rows"] == [[1], [2], [3], [], [4], [5]]


def test_cross_by_hand():
    q = np.zeros((3, 1, 2))
    k = np.zeros((3, 1, 2))
    v = np.array([[[1.0, 0.0]], [[3.0, 2.0]], [[9.0, 9.0]]])
    o, l = beam.cross(q, k, v, [0, 2, 3], [0, 3, 3], [2, 0])
    assert o[:, 0].tolist() == [[2, 1], [2, 1], [0, 0]]
    np.testing.assert_allclose(l[0], [math.log(2), math.log(2), -math.inf])
    o, _ = beam.cross(q, k, v, [0, 3], [0, 3], mask=[False, True, False])
    assert o[:, 0].tolist() == [[3, 2]] * 3
