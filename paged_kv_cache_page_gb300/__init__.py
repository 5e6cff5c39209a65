"""Paged KV-cache attention for GB300 (sm_103a): Python binding.

Thin ctypes layer over ``libpagedattn.so`` (``include/pagedattn.h``).  The
functions keep the C names and only marshal arguments (pointers, strides,
sizes, the current CUDA stream); every step of the computation runs in the
library's CUDA kernels.  PyTorch is used for device memory and streams: the
convenience arguments that are left as ``None`` (``out``, ``lse``,
``workspace``) are allocated with ``torch.empty`` on the tensors' device.

There is no CPU fallback: if the library has not been built (``python -m
paged_kv_cache_page_gb300.build``) or a tensor is not on a CUDA device, the
call raises.
"""

import ctypes
import math
import os

import torch

from .build import lib_path

PA_OK = 0
PA_ERR_INVALID_ARG = -1
PA_ERR_UNSUPPORTED = -2
PA_ERR_CUDA = -3
PA_ERR_WORKSPACE = -4
PA_F16 = 0
PA_BF16 = 1
PA_E4M3 = 2
PA_F32 = 3
PA_DEVERR_PAGE_OOB = 1
PA_DEVERR_LENGTH = 2
PA_DEVERR_TIMEOUT = 3
PA_DEVERR_CAPACITY = 4
PAGE_SIZE = 16
PA_NOALLOC_SCRATCH_BYTES = 8 << 20  # fixed split scratch of pa_fwd_kvcache_noalloc

_DTYPE = {torch.float16: PA_F16, torch.bfloat16: PA_BF16}


class PagedAttnError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"pagedattn error {code}: {msg}")
        self.code = code


class pa_tensor4(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_int64),
                ("stride_t", ctypes.c_int64), ("stride_h", ctypes.c_int64)]


_lib = None
_vp, _i32, _i64, _f32, _sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                              ctypes.c_size_t)

_SIGNATURES = {
    "pa_append_kv": (_i32, [pa_tensor4, pa_tensor4, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32,
                            _i32, _i32, _i32, _i64, _i32, _vp, _vp]),
    "pa_fwd_kvcache": (_i32, [_vp, _i64, _i64, _i64, pa_tensor4, pa_tensor4, _vp, _vp, _i32,
                              _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i64,
                              _i32, _f32, _i32, _i32, _vp, _vp, _vp, _sz, _vp, _i32, _vp]),
    "pa_fwd_kvcache_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32]),
    "pa_fwd_kvcache_rotary": (_i32, [_vp, _i64, _i64, _i64, pa_tensor4, pa_tensor4, _vp, _vp,
                                     _i32, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _i32,
                                     _i32, _i64, _i32, _vp, _vp, _i32, _i32, _i32, _f32, _i32,
                                     _i32, _vp, _vp, _vp, _sz, _vp, _i32, _vp]),
    "pa_fwd_kvcache_rotary_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                                   _i32]),
    "pa_fwd_kvcache_noalloc": (_i32, [_vp, _i64, _i64, _i64, pa_tensor4, pa_tensor4, _vp, _vp,
                                      _i32, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _i32,
                                      _i32, _i64, _i32, _f32, _i32, _i32, _vp, _vp, _vp, _i32,
                                      _vp]),
    "pa_fwd_varlen_unified": (_i32, [_vp, _i64, _i64, pa_tensor4, pa_tensor4, _vp, _vp, _vp,
                                     _i64, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                     _i64, _f32, _i32, _vp, _vp, _vp, _sz, _vp, _i32, _vp]),
    "pa_fwd_varlen_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32]),
    "pa_split_combine": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _i32,
                                _vp]),
    "pa_plan_step": (_i32, [_vp, _vp, _i32, _vp, _i64, _i32, _i32, _vp, _vp, _i64, _vp, _vp, _vp,
                            _vp, _i32, _vp, _vp, _vp]),
    "pa_release_pages": (_i32, [_vp, _vp, _i32, _vp, _i64, _i32, _i32, _vp, _vp, _i64, _vp, _vp,
                                _vp, _vp]),
    "pa_rotary_append_varlen": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64,
                                       _i64, pa_tensor4, pa_tensor4, _vp, _vp, _vp, _i32, _i64, _vp,
                                       _i64, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                       _i32, _i32, _i32, _i32, _i32, _vp, _vp]),
    "pa_fwd_varlen_e4m3": (_i32, [_vp, _i64, _i64, pa_tensor4, pa_tensor4, _vp, _vp, _vp, _vp, _vp,
                                  _i64, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i64,
                                  _f32, _i32, _vp, _vp, _vp, _sz, _vp, _i32, _vp]),
    "pa_fwd_varlen_e4m3_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32]),
    "pa_last_error_string": (ctypes.c_char_p, []),
    "pa_version": (_i32, []),
}


def load_library(path=None):
    """Load libpagedattn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with python -m paged_kv_cache_page_gb300.build")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(rc):
    if rc != PA_OK:
        raise PagedAttnError(rc, _lib.pa_last_error_string().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("pagedattn tensors must be on a CUDA device")


def _page_size(k_cache, block_table):
    """Tokens per page of a paged cache ``[num_pages, page_size, Hkv, D]``
    (ignored by the library for a contiguous cache)."""
    return k_cache.shape[1] if block_table is not None else PAGE_SIZE


def _stream(t):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _t4(cache):
    if cache.stride(-1) != 1:
        raise ValueError("cache head_dim axis must be contiguous")
    return pa_tensor4(cache.data_ptr(), cache.stride(0), cache.stride(1), cache.stride(2))


def _dtype(t):
    if t.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return _DTYPE[t.dtype]


def new_err_word(device):
    """int32[4] device error word (zeroed) for the ``err`` argument."""
    return torch.zeros(4, dtype=torch.int32, device=device)


def pa_append_kv(k_cache, v_cache, k_new, v_new, cache_seqlens, block_table=None, err=None):
    """Write k_new/v_new ``[B, Lnew, Hkv, D]`` at positions cache_seqlens[b] + i."""
    lib = load_library()
    _cuda(k_cache, v_cache, k_new, v_new, cache_seqlens, block_table)
    B, lnew, hkv, d = k_new.shape
    k_new = k_new.contiguous()
    v_new = v_new.contiguous()
    if block_table is not None:
        extent, max_pages, bt_stride = k_cache.shape[0], block_table.shape[1], block_table.stride(0)
    else:
        extent, max_pages, bt_stride = k_cache.shape[1], 0, 0
    _check(lib.pa_append_kv(_t4(k_cache), _t4(v_cache), _ptr(k_new), _ptr(v_new),
                            _ptr(cache_seqlens), _ptr(block_table), bt_stride, max_pages,
                            _page_size(k_cache, block_table), B, lnew, hkv, d, extent,
                            _dtype(k_cache), _ptr(err), _stream(k_cache)))


def fwd_kvcache_workspace_size(B, Lq, Hq, Hkv, D, max_seqlen_k, num_splits=0):
    return load_library().pa_fwd_kvcache_workspace_size(B, Lq, Hq, Hkv, D, max_seqlen_k,
                                                        num_splits)


def pa_fwd_kvcache(q, k_cache, v_cache, cache_seqlens, block_table=None, k=None, v=None,
                   scale=None, causal=False, num_splits=0, out=None, lse=None, workspace=None,
                   err=None, max_seqlen_k=None, return_lse=True, rotary_cos=None,
                   rotary_sin=None, rotary_interleaved=False):
    """flash_attn_with_kvcache-style forward; returns ``(out, lse)``.

    q ``[B, Lq, Hq, D]``; caches paged ``[num_pages, 16, Hkv, D]`` with
    ``block_table [B, max_pages]`` (int32) or contiguous ``[B, capacity, Hkv, D]``;
    ``k``/``v`` ``[B, Lnew, Hkv, D]`` are appended in the same call.
    ``max_seqlen_k`` defaults to the capacity implied by the table/cache shape.
    ``rotary_cos``/``rotary_sin`` ``[rotary_len, rotary_dim / 2]`` (q's dtype):
    rotary embedding of the new tokens' q and k (pa_fwd_kvcache_rotary).
    """
    lib = load_library()
    _cuda(q, k_cache, v_cache, cache_seqlens, block_table, k, v)
    B, lq, hq, d = q.shape
    hkv = k_cache.shape[2]
    lnew = 0 if k is None else k.shape[1]
    if k is not None:
        k = k.contiguous()
        v = v.contiguous()
    if block_table is not None:
        extent, max_pages, bt_stride = k_cache.shape[0], block_table.shape[1], block_table.stride(0)
        cap = max_pages * k_cache.shape[1]
    else:
        extent, max_pages, bt_stride = k_cache.shape[1], 0, 0
        cap = extent
    if max_seqlen_k is None:
        max_seqlen_k = cap
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, lq, hq, d), dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, hq, lq), dtype=torch.float32, device=q.device)
    if rotary_cos is not None:
        _cuda(rotary_cos, rotary_sin)
        rotary_cos = rotary_cos.contiguous()
        rotary_sin = rotary_sin.contiguous()
        ws_bytes = lib.pa_fwd_kvcache_rotary_workspace_size(B, lq, hq, hkv, d, lnew, max_seqlen_k,
                                                            num_splits)
        if workspace is None:
            workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
        ws_len = workspace.numel() * workspace.element_size()
        _check(lib.pa_fwd_kvcache_rotary(
            _ptr(q), q.stride(0), q.stride(1), q.stride(2), _t4(k_cache), _t4(v_cache), _ptr(k),
            _ptr(v), lnew, _ptr(cache_seqlens), _ptr(block_table), bt_stride, max_pages,
            _page_size(k_cache, block_table), B, lq, hq, hkv, d, extent, max_seqlen_k,
            _ptr(rotary_cos), _ptr(rotary_sin),
            rotary_cos.shape[0], 2 * rotary_cos.shape[1], int(bool(rotary_interleaved)),
            float(scale), int(bool(causal)), int(num_splits), _ptr(out), _ptr(lse),
            _ptr(workspace), ws_len, _ptr(err), _dtype(q), _stream(q)))
        return out, lse
    ws_bytes = lib.pa_fwd_kvcache_workspace_size(B, lq, hq, hkv, d, max_seqlen_k, num_splits)
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    ws_len = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.pa_fwd_kvcache(_ptr(q), q.stride(0), q.stride(1), q.stride(2), _t4(k_cache),
                              _t4(v_cache), _ptr(k), _ptr(v), lnew, _ptr(cache_seqlens),
                              _ptr(block_table), bt_stride, max_pages,
                              _page_size(k_cache, block_table), B, lq, hq, hkv, d, extent,
                              max_seqlen_k, float(scale), int(bool(causal)), int(num_splits),
                              _ptr(out), _ptr(lse), _ptr(workspace), ws_len, _ptr(err),
                              _dtype(q), _stream(q)))
    return out, lse


def pa_fwd_kvcache_noalloc(q, k_cache, v_cache, cache_seqlens, out, block_table=None, k=None,
                           v=None, lse=None, scale=None, causal=False, num_splits=0, err=None,
                           max_seqlen_k=None):
    """pa_fwd_kvcache for callers that cannot allocate device memory.

    The caller passes every tensor, including ``out`` (and optionally ``lse``);
    this wrapper allocates nothing and the library uses its own fixed split
    scratch (``PA_NOALLOC_SCRATCH_BYTES``).  Calls that could overlap on the GPU
    must be serialised by the caller because they share that scratch.
    """
    lib = load_library()
    _cuda(q, k_cache, v_cache, cache_seqlens, block_table, k, v, out, lse)
    B, lq, hq, d = q.shape
    hkv = k_cache.shape[2]
    lnew = 0 if k is None else k.shape[1]
    # the library reads k/v as contiguous [B, Lnew, Hkv, D]; a strided view
    # cannot be copied here (this call allocates nothing), so it is refused
    for name, t in (("k", k), ("v", v)):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"pa_fwd_kvcache_noalloc: {name} must be contiguous")
    if block_table is not None:
        extent, max_pages, bt_stride = k_cache.shape[0], block_table.shape[1], block_table.stride(0)
        cap = max_pages * k_cache.shape[1]
    else:
        extent, max_pages, bt_stride = k_cache.shape[1], 0, 0
        cap = extent
    if max_seqlen_k is None:
        max_seqlen_k = cap
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _check(lib.pa_fwd_kvcache_noalloc(_ptr(q), q.stride(0), q.stride(1), q.stride(2),
                                      _t4(k_cache), _t4(v_cache), _ptr(k), _ptr(v), lnew,
                                      _ptr(cache_seqlens), _ptr(block_table), bt_stride,
                                      max_pages, _page_size(k_cache, block_table), B, lq, hq, hkv,
                                      d, extent, max_seqlen_k,
                                      float(scale), int(bool(causal)), int(num_splits),
                                      _ptr(out), _ptr(lse), _ptr(err), _dtype(q), _stream(q)))
    return out, lse


def pa_fwd_varlen_unified(q, k_cache, v_cache, cu_seqlens_q, seqlens_k, block_table,
                          max_seqlen_q, max_seqlen_k, scale=None, causal=True, out=None, lse=None,
                          workspace=None, err=None, return_lse=True):
    """One launch over a mixed prefill/decode batch; returns ``(out, lse)``.

    q ``[total_q, Hq, D]`` packed by ``cu_seqlens_q [B+1]``; ``seqlens_k [B]``
    counts each sequence's keys including its new chunk (already in the cache).
    """
    lib = load_library()
    _cuda(q, k_cache, v_cache, cu_seqlens_q, seqlens_k, block_table)
    total_q, hq, d = q.shape
    hkv = k_cache.shape[2]
    B = cu_seqlens_q.numel() - 1
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((total_q, hq, d), dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((hq, total_q), dtype=torch.float32, device=q.device)
    ws_bytes = lib.pa_fwd_varlen_workspace_size(B, total_q, max_seqlen_q, hq, hkv, d,
                                                max_seqlen_k)
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    ws_len = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.pa_fwd_varlen_unified(_ptr(q), q.stride(0), q.stride(1), _t4(k_cache),
                                     _t4(v_cache), _ptr(cu_seqlens_q), _ptr(seqlens_k),
                                     _ptr(block_table), block_table.stride(0),
                                     block_table.shape[1], k_cache.shape[1], B, total_q,
                                     max_seqlen_q, max_seqlen_k,
                                     hq, hkv, d, k_cache.shape[0], float(scale),
                                     int(bool(causal)), _ptr(out), _ptr(lse), _ptr(workspace),
                                     ws_len, _ptr(err), _dtype(q), _stream(q)))
    return out, lse


def pa_split_combine(o_partial, lse_partial, out, lse=None, splits_per_seq=None):
    """Merge split partials: o_partial fp32 ``[S, B, Lq, Hq, D]``, lse_partial
    fp32 ``[S, B, Lq, Hq]`` into out ``[B, Lq, Hq, D]`` and lse ``[B, Hq, Lq]``."""
    lib = load_library()
    _cuda(o_partial, lse_partial, out, lse, splits_per_seq)
    S, B, lq, hq, d = o_partial.shape
    _check(lib.pa_split_combine(_ptr(o_partial.contiguous()), _ptr(lse_partial.contiguous()),
                                _ptr(splits_per_seq), S, B, lq, hq, d, _ptr(out), _ptr(lse),
                                _dtype(out), _stream(out)))
    return out, lse


# ---------------------------------------------------------------- a step over a paged cache
def _addr(t):
    return None if t is None else t.data_ptr()


def _want(name, t, dtype, dim, device, shape=None):
    """The argument's checks: on the call's CUDA device, of this type, number of axes (and shape),
    with a contiguous last axis."""
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on the call's CUDA device")
    if t.dtype is not dtype or t.dim() != dim or (shape is not None and tuple(t.shape) != shape):
        want = f"{dim}-d" if shape is None else str(shape)
        raise ValueError(f"{name} must be a {dtype} tensor, {want} (got {t.dtype}, {tuple(t.shape)})")
    if t.numel() > 1 and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return t.data_ptr()


def _run(fn, device, *args):
    """The library call on the tensors' device and its current stream."""
    stream = torch.cuda.current_stream(device).cuda_stream
    if device.index == torch.cuda.current_device():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc != PA_OK:
        _check(rc)


def pa_plan_step(cache_seqlens, q_lens, block_table, free_pages, free_count, page_size,
                 cu_seqlens_q=None, seqlens_k=None, slot_mapping=None, positions=None,
                 free_count_out=None, token_capacity=None, err=None):
    """Pages, block tables, slots and positions of a step's new tokens, from the lengths on the GPU;
    returns ``(cu_seqlens_q, seqlens_k, slot_mapping, positions)``.

    ``cache_seqlens``, ``q_lens`` int32 ``[B]``; ``block_table`` int32 ``[B, max_pages]`` (the new
    pages are written into it); ``free_pages`` int32 ``[num_pages]``, a stack of which the first
    ``free_count`` (int32 ``[1]``) are free.  ``free_count_out`` defaults to ``free_count`` itself.
    Outputs that are not given are allocated; ``slot_mapping`` (int64) and ``positions`` (int32)
    then hold ``token_capacity`` rows.
    """
    fn = (_lib or load_library()).pa_plan_step
    device = cache_seqlens.device
    i32 = torch.int32
    B = cache_seqlens.numel()
    if slot_mapping is None:
        if token_capacity is None:
            raise ValueError("pa_plan_step: token_capacity or slot_mapping must be given")
        slot_mapping = torch.empty(token_capacity, dtype=torch.int64, device=device)
    tokens = slot_mapping.numel()
    if token_capacity is not None and token_capacity != tokens:
        raise ValueError("pa_plan_step: slot_mapping does not have token_capacity rows")
    if cu_seqlens_q is None:
        cu_seqlens_q = torch.empty(B + 1, dtype=i32, device=device)
    if seqlens_k is None:
        seqlens_k = torch.empty(B, dtype=i32, device=device)
    if positions is None:
        positions = torch.empty(tokens, dtype=i32, device=device)
    if free_count_out is None:
        free_count_out = free_count
    table = _want("block_table", block_table, i32, 2, device)
    if block_table.shape[0] != B:
        raise ValueError("block_table must have a row for each sequence")
    _run(fn, device, _want("cache_seqlens", cache_seqlens, i32, 1, device),
         _want("q_lens", q_lens, i32, 1, device, (B,)), B, table, block_table.stride(0),
         block_table.shape[1], page_size, _want("free_pages", free_pages, i32, 1, device),
         _want("free_count", free_count, i32, 1, device, (1,)), free_pages.numel(),
         _want("cu_seqlens_q", cu_seqlens_q, i32, 1, device, (B + 1,)),
         _want("seqlens_k", seqlens_k, i32, 1, device, (B,)),
         _want("slot_mapping", slot_mapping, torch.int64, 1, device),
         _want("positions", positions, i32, 1, device, (tokens,)), tokens,
         _want("free_count_out", free_count_out, i32, 1, device, (1,)), _addr(err))
    return cu_seqlens_q, seqlens_k, slot_mapping, positions


def pa_release_pages(cache_seqlens, keep_lens, block_table, free_pages, free_count, page_size,
                     seqlens_out=None, free_count_out=None, err=None):
    """Gives the pages behind each sequence's first ``keep_lens[b]`` tokens back to the pool (0: the
    request has finished).  ``seqlens_out`` defaults to ``cache_seqlens`` itself, ``free_count_out``
    to ``free_count``; returns ``(seqlens_out, free_count_out)``."""
    fn = (_lib or load_library()).pa_release_pages
    device = cache_seqlens.device
    i32 = torch.int32
    B = cache_seqlens.numel()
    if seqlens_out is None:
        seqlens_out = cache_seqlens
    if free_count_out is None:
        free_count_out = free_count
    table = _want("block_table", block_table, i32, 2, device)
    if block_table.shape[0] != B:
        raise ValueError("block_table must have a row for each sequence")
    _run(fn, device, _want("cache_seqlens", cache_seqlens, i32, 1, device),
         _want("keep_lens", keep_lens, i32, 1, device, (B,)), B, table, block_table.stride(0),
         block_table.shape[1], page_size, _want("free_pages", free_pages, i32, 1, device),
         _want("free_count", free_count, i32, 1, device, (1,)), free_pages.numel(),
         _want("seqlens_out", seqlens_out, i32, 1, device, (B,)),
         _want("free_count_out", free_count_out, i32, 1, device, (1,)), _addr(err))
    return seqlens_out, free_count_out


_CACHE_DTYPE = {torch.float16: PA_F16, torch.bfloat16: PA_BF16, torch.float8_e4m3fn: PA_E4M3}


def _scale_addr(name, t, hkv, device):
    return None if t is None else _want(name, t, torch.float32, 1, device, (hkv,))


def pa_rotary_append_varlen(q, k, v, k_cache, v_cache, slot_mapping, positions=None,
                            rotary_cos=None, rotary_sin=None, rotary_interleaved=False,
                            pair_axis=None, k_scale=None, v_scale=None, q_out=None, err=None):
    """Rotates a ragged batch's q and k ``[T, H, D]`` and writes k and v into their cache slots;
    returns ``q_out``.

    Caches ``[num_pages, page_size, Hkv, D]`` of q's dtype or ``torch.float8_e4m3fn`` (with fp32
    scales ``k_scale``, ``v_scale`` ``[Hkv]``); ``slot_mapping`` int64 ``[T]``, negative for a token
    that is not stored.  ``positions`` int32 ``[T]`` or, with several axes, ``[n_axes, T]``, and
    ``pair_axis`` the axis of each of the ``rotary_dim / 2`` pairs (a sequence of ints).  Tables
    ``[rotary_len, rotary_dim / 2]`` in q's dtype or fp32; without them nothing is rotated.  ``q``
    may be ``None``; ``q_out`` may be ``q`` (in place).
    """
    fn = (_lib or load_library()).pa_rotary_append_varlen
    device = k.device
    dt = k.dtype
    if dt not in _DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    T, hkv, d = k.shape
    kp = _want("k", k, dt, 3, device)
    vp = _want("v", v, dt, 3, device, (T, hkv, d))
    qp = qo = None
    hq = q_st = q_sh = qo_st = qo_sh = 0
    if q is not None:
        hq = q.shape[1]
        qp = _want("q", q, dt, 3, device, (T, hq, d))
        if q_out is None:
            q_out = torch.empty((T, hq, d), dtype=dt, device=device)
        qo = _want("q_out", q_out, dt, 3, device, (T, hq, d))
        q_st, q_sh, qo_st, qo_sh = q.stride(0), q.stride(1), q_out.stride(0), q_out.stride(1)
    cdt = k_cache.dtype
    if cdt not in _CACHE_DTYPE:
        raise ValueError(f"unsupported cache dtype {cdt}")
    _want("k_cache", k_cache, cdt, 4, device)
    _want("v_cache", v_cache, cdt, 4, device, tuple(k_cache.shape))
    if k_cache.shape[2:] != (hkv, d):
        raise ValueError("the caches' heads and head_dim must be those of k")
    if cdt is not torch.float8_e4m3fn and (k_scale is not None or v_scale is not None):
        raise ValueError("k_scale and v_scale belong to e4m3 caches")
    pos = cos = sin = axes = None
    pos_stride = n_axes = rot_len = rot = rot_dt = 0
    if rotary_cos is not None:
        if positions is None or rotary_sin is None:
            raise ValueError("a rotation needs positions, rotary_cos and rotary_sin")
        many = positions.dim() == 2
        pos = _want("positions", positions, torch.int32, 2 if many else 1, device)
        if positions.shape[-1] != T:
            raise ValueError("positions must have a column for each token")
        n_axes, pos_stride = (positions.shape[0], positions.stride(0)) if many else (1, T)
        if many and n_axes == 1:
            pos_stride = T
        tdt = rotary_cos.dtype
        if tdt is not dt and tdt is not torch.float32:
            raise ValueError("the rotary tables must be of q's dtype or fp32")
        rot_dt = PA_F32 if tdt is torch.float32 else _DTYPE[dt]
        if not (rotary_cos.is_contiguous() and rotary_sin.is_contiguous()):
            raise ValueError("the rotary tables must be contiguous")
        cos = _want("rotary_cos", rotary_cos, tdt, 2, device)
        sin = _want("rotary_sin", rotary_sin, tdt, 2, device, tuple(rotary_cos.shape))
        rot_len, rot = rotary_cos.shape[0], 2 * rotary_cos.shape[1]
        if pair_axis is not None:
            axes = bytes(pair_axis)
            if len(axes) != rot // 2:
                raise ValueError("pair_axis must name an axis for each of the rotated pairs")
    _run(fn, device, qp, q_st, q_sh, kp, k.stride(0), k.stride(1), vp, v.stride(0), v.stride(1), qo,
         qo_st, qo_sh, _t4(k_cache), _t4(v_cache), _scale_addr("k_scale", k_scale, hkv, device),
         _scale_addr("v_scale", v_scale, hkv, device),
         _want("slot_mapping", slot_mapping, torch.int64, 1, device, (T,)), k_cache.shape[1],
         k_cache.shape[0], pos, pos_stride, n_axes, axes, cos, sin, rot_len, rot,
         int(bool(rotary_interleaved)), rot_dt, T, hq, hkv, d, _DTYPE[dt], _CACHE_DTYPE[cdt],
         _addr(err))
    return q_out


def fwd_varlen_e4m3_workspace_size(B, total_q, max_seqlen_q, Hq, Hkv, D, max_seqlen_k):
    return load_library().pa_fwd_varlen_e4m3_workspace_size(B, total_q, max_seqlen_q, Hq, Hkv, D,
                                                            max_seqlen_k)


def pa_fwd_varlen_e4m3(q, k_cache, v_cache, cu_seqlens_q, seqlens_k, block_table, max_seqlen_q,
                       max_seqlen_k, k_scale=None, v_scale=None, scale=None, causal=True, out=None,
                       lse=None, workspace=None, err=None, return_lse=True):
    """pa_fwd_varlen_unified over paged ``torch.float8_e4m3fn`` caches; returns ``(out, lse)``.

    ``k_scale``/``v_scale`` fp32 ``[Hkv]`` (device): what a stored value stands for is itself times
    its kv head's scale.  The other arguments are pa_fwd_varlen_unified's.
    """
    lib = _lib or load_library()
    device = q.device
    total_q, hq, d = q.shape
    qp = _want("q", q, q.dtype, 3, device)
    if q.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {q.dtype}")
    _want("k_cache", k_cache, torch.float8_e4m3fn, 4, device)
    _want("v_cache", v_cache, torch.float8_e4m3fn, 4, device, tuple(k_cache.shape))
    num_pages, page_size, hkv = k_cache.shape[:3]
    if k_cache.shape[3] != d:
        raise ValueError("the caches' head_dim must be that of q")
    B = seqlens_k.numel()
    table = _want("block_table", block_table, torch.int32, 2, device)
    if block_table.shape[0] != B:
        raise ValueError("block_table must have a row for each sequence")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((total_q, hq, d), dtype=q.dtype, device=device)
    elif not out.is_contiguous():
        raise ValueError("out must be contiguous")
    if lse is None:
        if return_lse:
            lse = torch.empty((hq, total_q), dtype=torch.float32, device=device)
    elif not lse.is_contiguous():
        raise ValueError("lse must be contiguous")
    if workspace is None:
        workspace = torch.empty(lib.pa_fwd_varlen_e4m3_workspace_size(
            B, total_q, max_seqlen_q, hq, hkv, d, max_seqlen_k), dtype=torch.uint8, device=device)
    _run(lib.pa_fwd_varlen_e4m3, device, qp, q.stride(0), q.stride(1), _t4(k_cache), _t4(v_cache),
         _scale_addr("k_scale", k_scale, hkv, device), _scale_addr("v_scale", v_scale, hkv, device),
         _want("cu_seqlens_q", cu_seqlens_q, torch.int32, 1, device, (B + 1,)),
         _want("seqlens_k", seqlens_k, torch.int32, 1, device), table, block_table.stride(0),
         block_table.shape[1], page_size, B, total_q, max_seqlen_q, max_seqlen_k, hq, hkv, d,
         num_pages, scale, 1 if causal else 0,
         _want("out", out, q.dtype, 3, device, (total_q, hq, d)),
         None if lse is None else _want("lse", lse, torch.float32, 2, device, (hq, total_q)),
         workspace.data_ptr(), workspace.numel() * workspace.element_size(), _addr(err),
         _DTYPE[q.dtype])
    return out, lse
