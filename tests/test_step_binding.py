"""The Python side of the serving-step calls, without a GPU: arguments on their way to the native
module."""

import pytest
import torch

import paged_kv_cache_page_gb300 as pa


class Recorder:
    def rotary_append_varlen(self, *a):
        self.axes = a[10]
        return 0


@pytest.fixture()
def native(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(pa, "_native", r)
    return r


def append(axes):
    x = torch.zeros(3, 2, 64, dtype=torch.float16)
    pa.pa_rotary_append_varlen(x, x, x, x, x, x, pair_axis=axes)


def test_pair_axis_is_any_sequence_of_ints(native):
    want = [0, 2, 1, 1]
    np = pytest.importorskip("numpy")
    for axes in (want, tuple(want), bytes(want), bytearray(want), range(4), np.array(want), np.array(want, "u1"),
                 np.array(want, ">i4"), torch.tensor(want), iter(want)):
        expected = list(range(4)) if isinstance(axes, range) else want
        append(axes)
        assert type(native.axes) is bytes and list(native.axes) == expected, axes
    append(None)
    assert native.axes is None
    append([])
    assert native.axes == b""


@pytest.mark.parametrize("axes", [4, 0, True, "0211", [0, 1.5], [0, -1], [0, 256], [[0, 1]], torch.tensor(4)])
def test_pair_axis_refusals(native, axes):
    with pytest.raises((TypeError, ValueError)):
        append(axes)
