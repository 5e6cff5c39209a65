"""Arguments that the serving-step calls refuse before any CUDA call (CPU)."""

import ctypes

import pytest
import torch

import paged_kv_cache_page_gb300 as pa
from paged_kv_cache_page_gb300 import build as pabuild


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.load_library()


P = 4096  # stands for an aligned device pointer; never read by a refused call


def plan(lib, **kw):
    a = dict(cached=P, new=P, B=2, table=P, bt=8, pages=8, ps=16, free=P, count=P, pool=64, cu=P,
             lens=P, slots=P, pos=P, cap=4, out=P, err=None)
    a.update(kw)
    return lib.pa_plan_step(*a.values(), None)


def release(lib, **kw):
    a = dict(cached=P, keep=P, B=2, table=P, bt=8, pages=8, ps=16, free=P, count=P, pool=64, lens=P,
             out=P, err=None)
    a.update(kw)
    return lib.pa_release_pages(*a.values(), None)


@pytest.mark.parametrize("call", [plan, release])
def test_step_refusals(lib, call):
    assert call(lib, B=-1) == pa.PA_ERR_INVALID_ARG
    assert call(lib, B=4097) == pa.PA_ERR_UNSUPPORTED
    for bad in (0, 8, 24, 48, 512):
        assert call(lib, ps=bad) == pa.PA_ERR_UNSUPPORTED
    assert call(lib, pages=0) == pa.PA_ERR_INVALID_ARG
    assert call(lib, bt=7) == pa.PA_ERR_INVALID_ARG
    assert call(lib, pages=1 << 30, bt=1 << 30) == pa.PA_ERR_UNSUPPORTED
    for bad in (0, -3, 1 << 31):
        assert call(lib, pool=bad) == pa.PA_ERR_INVALID_ARG
    for name in ("cached", "table", "free", "count", "lens", "out"):
        assert call(lib, **{name: None}) == pa.PA_ERR_INVALID_ARG, name
    assert lib.pa_last_error_string()


@pytest.mark.parametrize("call", [plan, release])
def test_step_sizes_near_2_31_are_refused(lib, call):
    """Places behind the last token, page or row of the largest step must fit in 32 bits."""
    pages = 1 << 27
    assert call(lib, pages=pages, bt=pages) == pa.PA_ERR_UNSUPPORTED
    assert call(lib, pages=pages - 255, bt=pages) == pa.PA_ERR_UNSUPPORTED
    assert call(lib, pool=(1 << 31) - (1 << 16) + 1) == pa.PA_ERR_INVALID_ARG


def test_plan_refusals(lib):
    assert plan(lib, cap=-1) == pa.PA_ERR_INVALID_ARG
    assert plan(lib, cap=(1 << 31) - (1 << 16) + 1) == pa.PA_ERR_UNSUPPORTED
    for name in ("new", "cu", "slots", "pos"):
        assert plan(lib, **{name: None}) == pa.PA_ERR_INVALID_ARG, name


def append(lib, axes=None, **kw):
    t4 = pa.pa_tensor4(P, 16 * 2 * 64, 2 * 64, 64)
    a = dict(q=P, q_st=512, q_sh=64, k=P, k_st=512, k_sh=64, v=P, v_st=512, v_sh=64, qo=P,
             qo_st=256, qo_sh=64, kc=t4, vc=t4, ks=None, vs=None, slots=P, ps=16, pool=8, pos=P,
             pos_st=5, n_axes=1, axes=axes, cos=P, sin=P, length=100, rot=64, inter=0,
             rdt=pa.PA_F16, T=5, Hq=4, Hkv=2, D=64, dtype=pa.PA_F16, cdt=pa.PA_F16, err=None)
    a.update(kw)
    return lib.pa_rotary_append_varlen(*a.values(), None)


def test_append_refusals(lib):
    bad4 = lambda **k: pa.pa_tensor4(*{**dict(p=P, b=2048, t=128, h=64), **k}.values())  # noqa: E731
    assert append(lib, T=0) == pa.PA_OK
    assert append(lib, T=-1) == pa.PA_ERR_INVALID_ARG
    assert append(lib, D=96) == pa.PA_ERR_UNSUPPORTED
    assert append(lib, dtype=pa.PA_E4M3) == pa.PA_ERR_UNSUPPORTED
    assert append(lib, cdt=pa.PA_BF16) == pa.PA_ERR_UNSUPPORTED
    assert append(lib, Hkv=0) == pa.PA_ERR_INVALID_ARG
    assert append(lib, Hq=0) == pa.PA_ERR_INVALID_ARG
    for bad in (bad4(p=None), bad4(p=P + 8), bad4(t=60), bad4(h=-64)):
        assert append(lib, kc=bad) == pa.PA_ERR_INVALID_ARG
        assert append(lib, vc=bad) == pa.PA_ERR_INVALID_ARG
    # 8-bit rows are 16-byte aligned in multiples of 16 elements
    assert append(lib, kc=bad4(t=72), cdt=pa.PA_E4M3) == pa.PA_ERR_INVALID_ARG
    for name in ("k", "v", "qo", "slots"):
        assert append(lib, **{name: None}) == pa.PA_ERR_INVALID_ARG, name
    for name in ("q_st", "k_sh", "v_st", "qo_sh"):
        assert append(lib, **{name: 36}) == pa.PA_ERR_INVALID_ARG, name
    assert append(lib, k=P + 8) == pa.PA_ERR_INVALID_ARG
    assert append(lib, ps=24) == pa.PA_ERR_UNSUPPORTED
    assert append(lib, pool=0) == pa.PA_ERR_INVALID_ARG
    for bad in (0, 7, 66):
        assert append(lib, rot=bad) == pa.PA_ERR_INVALID_ARG
    assert append(lib, length=0) == pa.PA_ERR_INVALID_ARG
    assert append(lib, rdt=pa.PA_BF16) == pa.PA_ERR_UNSUPPORTED
    assert append(lib, sin=None) == pa.PA_ERR_INVALID_ARG
    assert append(lib, pos=None) == pa.PA_ERR_INVALID_ARG
    assert append(lib, n_axes=5) == pa.PA_ERR_INVALID_ARG
    assert append(lib, n_axes=0) == pa.PA_ERR_INVALID_ARG
    assert append(lib, n_axes=2, pos_st=4) == pa.PA_ERR_INVALID_ARG
    assert append(lib, axes=bytes([0] * 31 + [1])) == pa.PA_ERR_INVALID_ARG
    assert "pair_axis[31]" in lib.pa_last_error_string().decode()


def attend(lib, **kw):
    t4 = pa.pa_tensor4(P, 16 * 2 * 64, 2 * 64, 64)
    a = dict(q=P, q_st=256, q_sh=64, kc=t4, vc=t4, ks=None, vs=None, cu=P, lens=P, table=P, bt=8,
             pages=8, ps=16, B=2, total=5, mq=4, mk=128, Hq=4, Hkv=2, D=64, pool=8, scale=0.125,
             causal=1, out=P, lse=None, ws=P, ws_bytes=1 << 30, err=None, dtype=pa.PA_F16)
    a.update(kw)
    return lib.pa_fwd_varlen_e4m3(*a.values(), None)


def test_attend_refusals(lib):
    t4 = lambda p=P, b=2048, t=128, h=64: pa.pa_tensor4(p, b, t, h)  # noqa: E731
    assert attend(lib, B=0) == pa.PA_OK
    assert attend(lib, total=0) == pa.PA_OK
    assert attend(lib, dtype=pa.PA_E4M3) == pa.PA_ERR_UNSUPPORTED
    assert attend(lib, D=256) == pa.PA_ERR_UNSUPPORTED
    assert attend(lib, Hq=3) == pa.PA_ERR_UNSUPPORTED
    assert attend(lib, Hkv=0) == pa.PA_ERR_INVALID_ARG
    for name in ("B", "total", "mq", "mk"):
        assert attend(lib, **{name: -1}) == pa.PA_ERR_INVALID_ARG, name
    assert attend(lib, B=4097) == pa.PA_ERR_UNSUPPORTED
    for bad in (t4(p=None), t4(p=P + 8), t4(t=72), t4(h=0)):
        assert attend(lib, kc=bad) == pa.PA_ERR_INVALID_ARG
        assert attend(lib, vc=bad) == pa.PA_ERR_INVALID_ARG
    for name in ("q", "cu", "lens", "table", "out"):
        assert attend(lib, **{name: None}) == pa.PA_ERR_INVALID_ARG, name
    assert attend(lib, q=P + 2) == pa.PA_ERR_INVALID_ARG
    assert attend(lib, q_sh=60) == pa.PA_ERR_INVALID_ARG
    assert attend(lib, pages=0) == pa.PA_ERR_INVALID_ARG
    assert attend(lib, bt=4) == pa.PA_ERR_INVALID_ARG
    assert attend(lib, ps=8) == pa.PA_ERR_UNSUPPORTED
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert attend(lib, scale=bad) == pa.PA_ERR_INVALID_ARG
    assert attend(lib, ws=None) == pa.PA_ERR_WORKSPACE
    assert attend(lib, ws_bytes=100) == pa.PA_ERR_WORKSPACE
    assert attend(lib, ws=P + 16) == pa.PA_ERR_WORKSPACE
    assert lib.pa_fwd_varlen_e4m3_workspace_size(2, 5, 4, 4, 2, 64, 128) > 0
    assert lib.pa_fwd_varlen_e4m3_workspace_size(0, 0, 0, 4, 2, 64, 128) == 0


def test_attend_sizes_near_2_31_are_refused(lib):
    pages = (1 << 27) - 255
    assert attend(lib, pages=pages, bt=pages) == pa.PA_ERR_UNSUPPORTED
    assert attend(lib, total=1 << 28, mq=1 << 28, mk=1 << 20) == pa.PA_ERR_UNSUPPORTED


def test_a_workspace_serves_smaller_batches(lib):
    size = lambda b, mq: lib.pa_fwd_varlen_e4m3_workspace_size(b, b * mq, mq, 4, 2, 64, 128)  # noqa: E731
    sizes = [[size(b, mq) for mq in (1, 24, 25, 32, 33, 500)] for b in (1, 31, 32, 4096)]
    for row in sizes:
        assert row == sorted(row)
    for column in zip(*sizes):
        assert list(column) == sorted(column)


def test_bindings_refuse_cpu_tensors(lib):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        pa.pa_plan_step(i(2), i(2), i(2, 4), i(8), i(1), 16, token_capacity=4)
    with pytest.raises(ValueError):
        pa.pa_plan_step(i(2), i(2), i(2, 4), i(8), i(1), 16)
    with pytest.raises(ValueError):
        pa.pa_release_pages(i(2), i(2), i(2, 4), i(8), i(1), 16)
    x = torch.zeros(3, 2, 64, dtype=torch.float16)
    c = torch.zeros(4, 16, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        pa.pa_rotary_append_varlen(x, x, x, c, c, torch.zeros(3, dtype=torch.int64))
    c8 = torch.zeros(4, 16, 2, 64, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        pa.pa_fwd_varlen_e4m3(x, c8, c8, i(2), i(1), i(1, 4), 3, 64)
    assert ctypes.sizeof(pa.pa_tensor4) == 32
