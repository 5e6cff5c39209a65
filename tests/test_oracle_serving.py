"""Pins of the serving-step oracle: worked examples and torch's own e4m3 conversion."""

import numpy as np
import torch

from oracle import serving as sv


def test_plan_worked_example():
    # pages of 16; request 0 fills its page, 1 starts, 2 rests, 3 does not fit
    r = sv.plan_step([15, 0, 5, 16], [2, 17, 0, 40], [[7, -1, -1, -1], [-1] * 4, [3, -1, -1, -1],
                                                       [4, -1, -1, -1]],
                     [9, 8, 1, 2, 0], 16, 60, 10)
    assert r["cu_seqlens_q"] == [0, 2, 19, 19, 19]
    assert r["seqlens_k"] == [17, 17, 5, 16]
    assert r["block_table"][0][:2] == [7, 0] and r["block_table"][1][:2] == [2, 1]
    assert r["slot_mapping"][:3] == [7 * 16 + 15, 0, 32]
    assert r["positions"][:3] == [15, 16, 0] and r["slot_mapping"][19:] == [-1] * 41
    assert r["free"] == [9, 8] and r["refused"] == [3] and r["bad"] == []


def test_release_worked_example():
    free, out, refused, bad = sv.release_pages([33, 20, 5, 40], [0, 17, 9, -1],
                                               [[4, 5, 6], [1, 2, -1], [3, -1, -1], [0, 7, 8]],
                                               [9], 16, 10)
    assert free == [9, 4, 5, 6] and out == [0, 17, 5, 40] and refused == [] and bad == [3]


def test_e4m3_matches_torch_on_every_value_and_midpoint():
    v = sv._e4m3_values()
    x = np.concatenate([v, (v[1:] + v[:-1]) / 2, v * 1.03, [500.0, 1e9]])
    x = np.concatenate([x, -x])
    want = torch.tensor(x, dtype=torch.float32).clamp(-448, 448).to(torch.float8_e4m3fn).double()
    assert np.array_equal(sv.e4m3(x.astype(np.float32)), want.numpy())
    assert np.isnan(sv.e4m3([np.nan])[0])


def test_rotary_axes_quarter_turns():
    cos, sin = np.array([[1.0, 1.0], [0.0, 0.0]]), np.array([[0.0, 0.0], [1.0, 1.0]])
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    # pair 0 on axis 0 (row 1: a quarter turn), pair 1 on axis 1 (row 0: none)
    y = sv.rotary_axes(x, cos, sin, [[1], [0]], [0, 1], False)
    assert y.ravel().tolist() == [-3.0, 2.0, 1.0, 4.0, 5.0, 6.0]
    y = sv.rotary_axes(x, cos, sin, [[0], [1]], [0, 1], True)
    assert y.ravel().tolist() == [1.0, 2.0, -4.0, 3.0, 5.0, 6.0]
    assert np.array_equal(sv.rotary_axes(x, cos, sin, [[0], [2]], [0, 1], True), x)
