"""Arguments that the beam search calls refuse before any CUDA call (CPU)."""

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


def select(lib, **kw):
    a = dict(x=P, sb=400, sk=100, scores=P, fin=None, end=-1, B=2, K=4, V=100, N=8, so=P, par=P, tok=P,
             fo=None, err=None, dtype=pa.PA_F16)
    a.update(kw)
    return lib.pa_beam_select(*a.values(), None)


def test_select_refusals(lib):
    assert select(lib, B=0) == pa.PA_OK
    assert select(lib, B=-1) == pa.PA_ERR_INVALID_ARG
    for name in ("K", "V", "N"):
        assert select(lib, **{name: 0}) == pa.PA_ERR_INVALID_ARG, name
    assert select(lib, K=33) == pa.PA_ERR_UNSUPPORTED
    assert select(lib, N=65) == pa.PA_ERR_UNSUPPORTED
    assert select(lib, V=(1 << 24) + 1) == pa.PA_ERR_UNSUPPORTED
    assert select(lib, B=(1 << 20) + 1) == pa.PA_ERR_UNSUPPORTED
    for bad in (pa.PA_E4M3, -1, 7):
        assert select(lib, dtype=bad) == pa.PA_ERR_UNSUPPORTED
    for name in ("x", "scores", "so", "par", "tok"):
        assert select(lib, **{name: None}) == pa.PA_ERR_INVALID_ARG, name
    assert select(lib, x=P + 1) == pa.PA_ERR_INVALID_ARG
    assert select(lib, x=P + 2, dtype=pa.PA_F32) == pa.PA_ERR_INVALID_ARG
    assert select(lib, sk=-1) == pa.PA_ERR_INVALID_ARG
    assert select(lib, sb=-1) == pa.PA_ERR_INVALID_ARG
    assert select(lib, end=100) == pa.PA_ERR_INVALID_ARG
    assert select(lib, fin=P) == pa.PA_ERR_INVALID_ARG
    assert lib.pa_last_error_string()


def test_select_refuses_to_replace_its_inputs(lib):
    assert select(lib, so=P) == pa.PA_ERR_INVALID_ARG
    assert b"replaced" in lib.pa_last_error_string()
    assert select(lib, so=2 * P, fin=P, fo=P, end=3) == pa.PA_ERR_INVALID_ARG
    assert b"replaced" in lib.pa_last_error_string()


def reorder(lib, **kw):
    a = dict(par=P, lens=P, B=2, K=4, table=P, bt=8, pages=8, ps=16, free=P, count=P, pool=64, out=P, bto=8,
             lo=P, copies=P, co=P, err=None)
    a.update(kw)
    return lib.pa_beam_reorder(*a.values(), None)


def test_reorder_refusals(lib):
    assert reorder(lib, B=-1) == pa.PA_ERR_INVALID_ARG
    assert reorder(lib, K=0) == pa.PA_ERR_INVALID_ARG
    assert reorder(lib, K=33) == pa.PA_ERR_UNSUPPORTED
    assert reorder(lib, B=1025) == pa.PA_ERR_UNSUPPORTED
    for bad in (0, 8, 24, 48, 512):
        assert reorder(lib, ps=bad) == pa.PA_ERR_UNSUPPORTED
    for bad in (dict(pages=0), dict(bt=7), dict(bto=7), dict(pool=0), dict(pool=1 << 31), dict(bt=9)):
        assert reorder(lib, **bad) == pa.PA_ERR_INVALID_ARG, bad
    # another table may have another stride
    assert reorder(lib, bt=9, out=2 * P, par=None) == pa.PA_ERR_INVALID_ARG
    wide = (1 << 27) - 255
    assert reorder(lib, pages=wide, bt=wide, bto=wide) == pa.PA_ERR_UNSUPPORTED
    assert reorder(lib, B=1024, pages=1 << 22, bt=1 << 22, bto=1 << 22) == pa.PA_ERR_UNSUPPORTED
    for name in ("par", "lens", "table", "free", "count", "out", "lo", "copies", "co"):
        assert reorder(lib, **{name: None}) == pa.PA_ERR_INVALID_ARG, name


def copy(lib, caches=(P, P), **kw):
    a = dict(copies=P, n=3, caches=(ctypes.c_void_p * len(caches))(*caches), n_caches=len(caches),
             sb=16 * 128, st=128, sh=64, hb=64, H=2, ps=16, pool=9, err=None)
    a.update(kw)
    return lib.pa_copy_pages(*a.values(), None)


def test_copy_refusals(lib):
    assert copy(lib, n=0) == pa.PA_OK
    assert copy(lib, n_caches=0) == pa.PA_OK
    for bad in (dict(n=-1), dict(n_caches=-1), dict(H=0), dict(ps=0), dict(pool=0), dict(hb=0),
                dict(hb=24), dict(sb=8), dict(st=-16), dict(sh=40), dict(copies=None)):
        assert copy(lib, **bad) == pa.PA_ERR_INVALID_ARG, bad
    assert copy(lib, caches=(P, None)) == pa.PA_ERR_INVALID_ARG
    assert copy(lib, caches=(P, P + 8)) == pa.PA_ERR_INVALID_ARG
    assert copy(lib, pool=1 << 31) == pa.PA_ERR_UNSUPPORTED
    assert copy(lib, ps=1 << 28, H=1 << 10) == pa.PA_ERR_UNSUPPORTED


def cross(lib, **kw):
    a = dict(q=P, q_st=256, q_sh=64, k=P, k_st=256, k_sh=64, v=P, v_st=256, v_sh=64, cu_q=P, cu_k=P,
             lens=None, mask=None, B=2, tq=5, tk=50, mq=4, mk=40, Hq=4, Hkv=2, D=64, scale=0.125, out=P,
             lse=None, ws=None, ws_bytes=0, err=None, dtype=pa.PA_F16)
    a.update(kw)
    return lib.pa_fwd_cross(*a.values(), None)


def test_cross_refusals(lib):
    for name in ("B", "tq", "mq"):
        assert cross(lib, **{name: 0}) == pa.PA_OK, name
    for name in ("B", "tq", "tk", "mq", "mk"):
        assert cross(lib, **{name: -1}) == pa.PA_ERR_INVALID_ARG, name
    assert cross(lib, dtype=pa.PA_E4M3) == pa.PA_ERR_UNSUPPORTED
    for bad in (32, 96, 256):
        assert cross(lib, D=bad) == pa.PA_ERR_UNSUPPORTED
    assert cross(lib, Hq=3) == pa.PA_ERR_UNSUPPORTED
    assert cross(lib, Hkv=0) == pa.PA_ERR_INVALID_ARG
    for name in ("q", "k", "v", "cu_q", "cu_k", "out"):
        assert cross(lib, **{name: None}) == pa.PA_ERR_INVALID_ARG, name
    for name in ("q", "k", "v", "out"):
        assert cross(lib, **{name: P + 8}) == pa.PA_ERR_INVALID_ARG, name
    for name in ("q_st", "q_sh", "k_st", "k_sh", "v_st", "v_sh"):
        for bad in (0, 36, -64):
            assert cross(lib, **{name: bad}) == pa.PA_ERR_INVALID_ARG, name
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert cross(lib, scale=bad) == pa.PA_ERR_INVALID_ARG
    assert cross(lib, tq=2 ** 31 - 1) == pa.PA_ERR_UNSUPPORTED
    assert cross(lib, tk=2 ** 31 - 1) == pa.PA_ERR_UNSUPPORTED
    assert cross(lib, B=1 << 20, tq=1 << 30, mq=1 << 20) == pa.PA_ERR_UNSUPPORTED
    wide = dict(tq=1 << 28, tk=1 << 28, mq=1 << 28, mk=1 << 28, ws=P, ws_bytes=1 << 40)
    assert cross(lib, **wide) == pa.PA_ERR_UNSUPPORTED
    # many rows need a workspace
    size = lib.pa_fwd_cross_workspace_size(500, 400, 4, 2, 64)
    assert size > 0 and lib.pa_fwd_cross_workspace_size(5, 4, 4, 2, 64) == 0
    many = dict(tq=500, mq=400, ws=P, ws_bytes=size)
    for bad in (dict(ws=None), dict(ws=P + 16), dict(ws_bytes=size - 1)):
        assert cross(lib, **{**many, **bad}) == pa.PA_ERR_WORKSPACE, bad


def test_bindings_refuse_cpu_tensors():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    x = torch.zeros(3, 2, 64, dtype=torch.float16)
    for call in (lambda: pa.pa_beam_select(torch.zeros(1, 2, 9), torch.zeros(1, 2)),
                 lambda: pa.pa_beam_reorder(i(1, 2), i(2), i(2, 4), i(8), i(1), 16),
                 lambda: pa.pa_copy_pages(i(2, 3), [torch.zeros(4, 16, 2, 64)]),
                 lambda: pa.pa_fwd_cross(x, x, x, i(2), i(2), 3, 3)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        pa.pa_beam_select(torch.zeros(1, 2, 9), torch.zeros(1, 2), 4, parents=i(1, 3))
