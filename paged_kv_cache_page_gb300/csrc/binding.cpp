// Python module `_binding`: the serving-step calls (pa_plan_step,
// pa_release_pages, pa_rotary_append_varlen, pa_fwd_varlen_e4m3; pa_beam_select,
// pa_beam_reorder, pa_copy_pages, pa_fwd_cross) from torch tensors.  A decode step's kernels take 4 to 6 us, and checking a dozen tensors
// and packing forty ctypes arguments from Python took 16 to 32 us a call on the
// GB300's host cores; here a call takes 3 to 5 us, its launch included.  The
// module holds no computation: it checks types, shapes and devices, and calls
// the C ABI on the tensors' device and its current stream, without the
// interpreter's lock: a launch waits where the queue of launches is full.
//
// The entry points are given as addresses by bind(), so that the module works
// with whichever libpagedattn.so has been loaded.  Each function returns the
// library's return code (0: done); a bad argument raises ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/pagedattn.h"

namespace {

struct Entries {
  decltype(&pa_plan_step) plan = nullptr;
  decltype(&pa_release_pages) release = nullptr;
  decltype(&pa_rotary_append_varlen) append = nullptr;
  decltype(&pa_fwd_varlen_e4m3) attend = nullptr;
  decltype(&pa_fwd_varlen_e4m3_workspace_size) attend_workspace = nullptr;
  decltype(&pa_beam_select) select = nullptr;
  decltype(&pa_beam_reorder) reorder = nullptr;
  decltype(&pa_copy_pages) copy = nullptr;
  decltype(&pa_fwd_cross) cross = nullptr;
  decltype(&pa_fwd_cross_workspace_size) cross_workspace = nullptr;
} g_entries;

struct BadArgument : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct PythonError {};  // the interpreter's error is set

[[noreturn]] void bad(const char* name, const std::string& what) {
  throw BadArgument(std::string(name) + " " + what);
}

const at::Tensor& tensor_of(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad(name, "must be a tensor");
  return THPVariable_Unpack(o);
}

// The device of a call: that of its first tensor, a CUDA one.
c10::Device device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) bad(name, "must be on a CUDA device");
  return t.device();
}

// The checks of an argument; -1 in `shape` stands for any size.  The last axis
// is contiguous.
const at::Tensor& want(PyObject* o, const char* name, at::ScalarType type, c10::Device device,
                       std::initializer_list<int64_t> shape) {
  const at::Tensor& t = tensor_of(o, name);
  if (!t.is_cuda() || t.device() != device) bad(name, "must be on the call's CUDA device");
  bool ok = t.scalar_type() == type && t.dim() == (int64_t)shape.size();
  if (ok) {
    int64_t i = 0;
    for (int64_t n : shape) {
      ok = ok && (n < 0 || t.size(i) == n);
      ++i;
    }
  }
  if (!ok) {
    std::string s = "must be a ";
    s += c10::toString(type);
    s += " tensor of shape (";
    for (int64_t n : shape) s += (n < 0 ? std::string("*") : std::to_string(n)) + ", ";
    bad(name, s + ")");
  }
  const int64_t last = t.dim() - 1;
  if (t.numel() > 1 && t.size(last) > 1 && t.stride(last) != 1)
    bad(name, "must have a contiguous last axis");
  return t;
}
template <typename P>
P* ptr(const at::Tensor& t) {
  return reinterpret_cast<P*>(t.data_ptr());
}
int32_t* err_of(PyObject* o, c10::Device device) {
  return o == Py_None ? nullptr : ptr<int32_t>(want(o, "err", at::kInt, device, {4}));
}

long long integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw PythonError();
  return x;
}
int int_of(PyObject* o, const char* name) {
  const long long x = integer(o);
  if (x < -2147483648LL || x > 2147483647LL) bad(name, "does not fit in 32 bits");
  return (int)x;
}
int size_of(int64_t x, const char* name) {
  if (x > 2147483647LL) bad(name, "is too large");
  return (int)x;
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw PythonError();
  return x != 0;
}

int dtype_of(at::ScalarType t) {
  return t == at::kHalf ? PA_F16 : t == at::kBFloat16 ? PA_BF16 : -1;
}

pa_stream_t stream_of(c10::Device device) {
  return reinterpret_cast<pa_stream_t>(
      c10::cuda::getCurrentCUDAStream(device.index()).stream());
}

pa_tensor4 cache_view(const at::Tensor& t) {
  return pa_tensor4{t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const PythonError&) {
  } catch (const BadArgument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// fn(args...) without the interpreter's lock, and its return code.  The caller's
// references keep the tensors alive.
template <typename F, typename... A>
PyObject* unlocked(F fn, A... args) {
  PyThreadState* const state = PyEval_SaveThread();
  const int rc = fn(args...);
  PyEval_RestoreThread(state);
  return PyLong_FromLong(rc);
}

bool count_is(Py_ssize_t n, Py_ssize_t expected) {
  if (n == expected) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", expected, n);
  return false;
}

uintptr_t address_of(PyObject* o) { return (uintptr_t)(unsigned long long)integer(o); }
template <typename F>
void entry(F& f, PyObject* address) {
  f = reinterpret_cast<F>(address_of(address));
}

// bind(plan, release, append, attend, attend_workspace): entry addresses
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    entry(g_entries.plan, a[0]);
    entry(g_entries.release, a[1]);
    entry(g_entries.append, a[2]);
    entry(g_entries.attend, a[3]);
    entry(g_entries.attend_workspace, a[4]);
    Py_RETURN_NONE;
  });
}

// bind_beam(select, reorder, copy, cross, cross_workspace): entry addresses
PyObject* bind_beam(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    entry(g_entries.select, a[0]);
    entry(g_entries.reorder, a[1]);
    entry(g_entries.copy, a[2]);
    entry(g_entries.cross, a[3]);
    entry(g_entries.cross_workspace, a[4]);
    Py_RETURN_NONE;
  });
}

// plan_step(cache_seqlens, q_lens, block_table, free_pages, free_count, page_size,
//           cu_seqlens_q, seqlens_k, slot_mapping, positions, free_count_out, err)
PyObject* plan_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 12)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& lens = tensor_of(a[0], "cache_seqlens");
    const c10::Device device = device_of(lens, "cache_seqlens");
    const int64_t B = lens.numel();
    const auto& table = want(a[2], "block_table", at::kInt, device, {B, -1});
    const auto& pool = want(a[3], "free_pages", at::kInt, device, {-1});
    const auto& slots = want(a[8], "slot_mapping", at::kLong, device, {-1});
    const int64_t rows = slots.numel();
    const c10::cuda::CUDAGuard guard(device);
    return unlocked(
        g_entries.plan,
        ptr<int32_t>(want(a[0], "cache_seqlens", at::kInt, device, {B})),
        ptr<int32_t>(want(a[1], "q_lens", at::kInt, device, {B})), size_of(B, "the batch"),
        ptr<int32_t>(table), table.stride(0), size_of(table.size(1), "block_table"),
        int_of(a[5], "page_size"), ptr<int32_t>(pool),
        ptr<int32_t>(want(a[4], "free_count", at::kInt, device, {1})), pool.numel(),
        ptr<int32_t>(want(a[6], "cu_seqlens_q", at::kInt, device, {B + 1})),
        ptr<int32_t>(want(a[7], "seqlens_k", at::kInt, device, {B})), ptr<int64_t>(slots),
        ptr<int32_t>(want(a[9], "positions", at::kInt, device, {rows})),
        size_of(rows, "slot_mapping"),
        ptr<int32_t>(want(a[10], "free_count_out", at::kInt, device, {1})), err_of(a[11], device),
        stream_of(device));
  });
}

// release_pages(cache_seqlens, keep_lens, block_table, free_pages, free_count, page_size,
//               seqlens_out, free_count_out, err)
PyObject* release_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& lens = tensor_of(a[0], "cache_seqlens");
    const c10::Device device = device_of(lens, "cache_seqlens");
    const int64_t B = lens.numel();
    const auto& table = want(a[2], "block_table", at::kInt, device, {B, -1});
    const auto& pool = want(a[3], "free_pages", at::kInt, device, {-1});
    const c10::cuda::CUDAGuard guard(device);
    return unlocked(
        g_entries.release,
        ptr<int32_t>(want(a[0], "cache_seqlens", at::kInt, device, {B})),
        ptr<int32_t>(want(a[1], "keep_lens", at::kInt, device, {B})), size_of(B, "the batch"),
        ptr<int32_t>(table), table.stride(0), size_of(table.size(1), "block_table"),
        int_of(a[5], "page_size"), ptr<int32_t>(pool),
        ptr<int32_t>(want(a[4], "free_count", at::kInt, device, {1})), pool.numel(),
        ptr<int32_t>(want(a[6], "seqlens_out", at::kInt, device, {B})),
        ptr<int32_t>(want(a[7], "free_count_out", at::kInt, device, {1})), err_of(a[8], device),
        stream_of(device));
  });
}

const float* scale_of(PyObject* o, const char* name, int64_t heads, c10::Device device) {
  return o == Py_None ? nullptr : ptr<float>(want(o, name, at::kFloat, device, {heads}));
}

// rotary_append_varlen(q, k, v, k_cache, v_cache, slot_mapping, positions, cos, sin, interleaved,
//                      pair_axis, k_scale, v_scale, q_out, err)
PyObject* rotary_append_varlen(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 15)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& k = tensor_of(a[1], "k");
    const c10::Device device = device_of(k, "k");
    const at::ScalarType type = k.scalar_type();
    const int dtype = dtype_of(type);
    if (dtype < 0 || k.dim() != 3) bad("k", "must be a 3-d fp16 or bf16 tensor");
    const int64_t T = k.size(0), hkv = k.size(1), d = k.size(2);
    want(a[1], "k", type, device, {T, hkv, d});
    const auto& v = want(a[2], "v", type, device, {T, hkv, d});
    const void* qp = nullptr;
    void* qo = nullptr;
    int64_t hq = 0, q_st = 0, q_sh = 0, qo_st = 0, qo_sh = 0;
    if (a[0] != Py_None) {
      const auto& q = want(a[0], "q", type, device, {T, -1, d});
      hq = q.size(1);
      const auto& out = want(a[13], "q_out", type, device, {T, hq, d});
      qp = q.data_ptr();
      qo = out.data_ptr();
      q_st = q.stride(0);
      q_sh = q.stride(1);
      qo_st = out.stride(0);
      qo_sh = out.stride(1);
    }
    const at::ScalarType held = tensor_of(a[3], "k_cache").scalar_type();
    const bool e4m3 = held == at::kFloat8_e4m3fn;
    if (!e4m3 && held != type) bad("k_cache", "must hold the type of k or float8_e4m3fn");
    const auto& kc = want(a[3], "k_cache", held, device, {-1, -1, hkv, d});
    const auto& vc = want(a[4], "v_cache", held, device, {kc.size(0), kc.size(1), hkv, d});
    if (!e4m3 && (a[11] != Py_None || a[12] != Py_None))
      bad("k_scale and v_scale", "belong to e4m3 caches");
    const auto& slots = want(a[5], "slot_mapping", at::kLong, device, {T});
    const void *cos = nullptr, *sin = nullptr;
    const int32_t* pos = nullptr;
    const uint8_t* axes = nullptr;
    int64_t pos_stride = T, n_axes = 1, rot_len = 0, rot = 0;
    int rot_type = dtype;
    if (a[7] != Py_None) {
      if (a[6] == Py_None || a[8] == Py_None)
        bad("a rotation", "needs positions, rotary_cos and rotary_sin");
      const auto& c = tensor_of(a[7], "rotary_cos");
      const at::ScalarType tt = c.scalar_type();
      if (tt != type && tt != at::kFloat) bad("rotary_cos", "must be of q's type or fp32");
      want(a[7], "rotary_cos", tt, device, {-1, -1});
      const auto& s = want(a[8], "rotary_sin", tt, device, {c.size(0), c.size(1)});
      if (!c.is_contiguous() || !s.is_contiguous()) bad("the rotary tables", "must be contiguous");
      rot_type = tt == at::kFloat ? PA_F32 : dtype;
      cos = c.data_ptr();
      sin = s.data_ptr();
      rot_len = c.size(0);
      rot = 2 * c.size(1);
      const auto& p = tensor_of(a[6], "positions");
      if (p.dim() == 2) {
        want(a[6], "positions", at::kInt, device, {-1, T});
        n_axes = p.size(0);
        if (n_axes > 1) pos_stride = p.stride(0);
      } else {
        want(a[6], "positions", at::kInt, device, {T});
      }
      pos = ptr<int32_t>(p);
      if (a[10] != Py_None) {
        char* data = nullptr;
        Py_ssize_t size = 0;
        if (PyBytes_AsStringAndSize(a[10], &data, &size) < 0) throw PythonError();
        if (size != rot / 2) bad("pair_axis", "must name an axis for each of the rotated pairs");
        axes = reinterpret_cast<const uint8_t*>(data);
      }
    }
    const c10::cuda::CUDAGuard guard(device);
    return unlocked(
        g_entries.append,
        qp, q_st, q_sh, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0),
        v.stride(1), qo, qo_st, qo_sh, cache_view(kc), cache_view(vc),
        scale_of(a[11], "k_scale", hkv, device), scale_of(a[12], "v_scale", hkv, device),
        ptr<int64_t>(slots), size_of(kc.size(1), "the page size"), kc.size(0), pos, pos_stride,
        size_of(n_axes, "positions"), axes, cos, sin, size_of(rot_len, "rotary_cos"),
        size_of(rot, "rotary_cos"), truth(a[9]) ? 1 : 0, rot_type, size_of(T, "k"),
        size_of(hq, "q"), size_of(hkv, "k"), size_of(d, "k"), dtype, e4m3 ? PA_E4M3 : dtype,
        err_of(a[14], device), stream_of(device));
  });
}

// fwd_varlen_e4m3(q, k_cache, v_cache, cu_seqlens_q, seqlens_k, block_table, max_seqlen_q,
//                 max_seqlen_k, k_scale, v_scale, scale, causal, out, lse, workspace, err)
PyObject* fwd_varlen_e4m3(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 16)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& q = tensor_of(a[0], "q");
    const c10::Device device = device_of(q, "q");
    const int dtype = dtype_of(q.scalar_type());
    if (dtype < 0 || q.dim() != 3) bad("q", "must be a 3-d fp16 or bf16 tensor");
    const int64_t rows = q.size(0), hq = q.size(1), d = q.size(2);
    want(a[0], "q", q.scalar_type(), device, {rows, hq, d});
    const auto& kc = want(a[1], "k_cache", at::kFloat8_e4m3fn, device, {-1, -1, -1, d});
    const int64_t pages = kc.size(0), page = kc.size(1), hkv = kc.size(2);
    const auto& vc = want(a[2], "v_cache", at::kFloat8_e4m3fn, device, {pages, page, hkv, d});
    const auto& lens = want(a[4], "seqlens_k", at::kInt, device, {-1});
    const int64_t B = lens.numel();
    const auto& cu = want(a[3], "cu_seqlens_q", at::kInt, device, {B + 1});
    const auto& table = want(a[5], "block_table", at::kInt, device, {B, -1});
    const auto& out = want(a[12], "out", q.scalar_type(), device, {rows, hq, d});
    if (!out.is_contiguous()) bad("out", "must be contiguous");
    float* lse = nullptr;
    if (a[13] != Py_None) {
      const auto& l = want(a[13], "lse", at::kFloat, device, {hq, rows});
      if (!l.is_contiguous()) bad("lse", "must be contiguous");
      lse = ptr<float>(l);
    }
    const int max_q = int_of(a[6], "max_seqlen_q"), max_k = int_of(a[7], "max_seqlen_k");
    double scale = 0;
    if (a[10] == Py_None) {
      scale = 1.0 / std::sqrt((double)d);
    } else {
      scale = PyFloat_AsDouble(a[10]);
      if (scale == -1.0 && PyErr_Occurred()) throw PythonError();
    }
    const c10::cuda::CUDAGuard guard(device);
    at::Tensor scratch;
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (a[14] != Py_None) {
      const at::Tensor& w = tensor_of(a[14], "workspace");
      if (!w.is_cuda() || w.device() != device || !w.is_contiguous())
        bad("workspace", "must be contiguous, on the call's CUDA device");
      ws = w.data_ptr();
      ws_bytes = (size_t)w.numel() * w.element_size();
    } else {
      ws_bytes = g_entries.attend_workspace(size_of(B, "the batch"), size_of(rows, "q"), max_q,
                                            size_of(hq, "q"), size_of(hkv, "k_cache"),
                                            size_of(d, "q"), max_k);
      scratch = at::empty({(int64_t)ws_bytes}, q.options().dtype(at::kByte));
      ws = scratch.data_ptr();
    }
    return unlocked(
        g_entries.attend,
        q.data_ptr(), q.stride(0), q.stride(1), cache_view(kc), cache_view(vc),
        scale_of(a[8], "k_scale", hkv, device), scale_of(a[9], "v_scale", hkv, device),
        ptr<int32_t>(cu), ptr<int32_t>(lens), ptr<int32_t>(table), table.stride(0),
        size_of(table.size(1), "block_table"), size_of(page, "the page size"),
        size_of(B, "the batch"), size_of(rows, "q"), max_q, max_k, size_of(hq, "q"),
        size_of(hkv, "k_cache"), size_of(d, "q"), pages, (float)scale, truth(a[11]) ? 1 : 0,
        out.data_ptr(), lse, ws, ws_bytes, err_of(a[15], device), dtype, stream_of(device));
  });
}

// A contiguous tensor of flags, one byte each.
uint8_t* flags_of(PyObject* o, const char* name, c10::Device device,
                  std::initializer_list<int64_t> shape) {
  if (o == Py_None) return nullptr;
  const at::ScalarType type = tensor_of(o, name).scalar_type();
  const auto& t = want(o, name, type == at::kByte ? at::kByte : at::kBool, device, shape);
  if (!t.is_contiguous()) bad(name, "must be contiguous");
  return ptr<uint8_t>(t);
}
template <typename T>
T* dense(PyObject* o, const char* name, at::ScalarType type, c10::Device device,
         std::initializer_list<int64_t> shape) {
  const auto& t = want(o, name, type, device, shape);
  if (!t.is_contiguous()) bad(name, "must be contiguous");
  return ptr<T>(t);
}

// beam_select(logits, scores, finished, end_token, scores_out, parents, tokens, finished_out, err)
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& x = tensor_of(a[0], "logits");
    const c10::Device device = device_of(x, "logits");
    const at::ScalarType type = x.scalar_type();
    const int dtype = type == at::kFloat ? PA_F32 : dtype_of(type);
    if (dtype < 0 || x.dim() != 3) bad("logits", "must be a 3-d fp16, bf16 or fp32 tensor");
    const int64_t B = x.size(0), K = x.size(1), V = x.size(2);
    want(a[0], "logits", type, device, {B, K, V});
    const auto& parents = want(a[5], "parents", at::kInt, device, {B, -1});
    const int64_t N = parents.size(1);
    const c10::cuda::CUDAGuard guard(device);
    return unlocked(
        g_entries.select, x.data_ptr(), x.stride(0), x.stride(1),
        dense<float>(a[1], "scores", at::kFloat, device, {B, K}),
        flags_of(a[2], "finished", device, {B, K}), int_of(a[3], "end_token"),
        size_of(B, "the batch"), size_of(K, "the beams"), size_of(V, "the vocabulary"),
        size_of(N, "parents"), dense<float>(a[4], "scores_out", at::kFloat, device, {B, N}),
        dense<int32_t>(a[5], "parents", at::kInt, device, {B, N}),
        dense<int32_t>(a[6], "tokens", at::kInt, device, {B, N}),
        flags_of(a[7], "finished_out", device, {B, N}), err_of(a[8], device), dtype,
        stream_of(device));
  });
}

// beam_reorder(parents, seqlens, block_table, free_pages, free_count, page_size, block_table_out,
//              seqlens_out, copies, free_count_out, err)
PyObject* beam_reorder(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& parents = tensor_of(a[0], "parents");
    const c10::Device device = device_of(parents, "parents");
    if (parents.dim() != 2) bad("parents", "must be a 2-d tensor");
    const int64_t B = parents.size(0), K = parents.size(1), rows = B * K;
    const auto& table = want(a[2], "block_table", at::kInt, device, {rows, -1});
    const int64_t width = table.size(1);
    const auto& out = want(a[6], "block_table_out", at::kInt, device, {rows, width});
    const auto& pool = want(a[3], "free_pages", at::kInt, device, {-1});
    // (a table of one row: its stride does not matter)
    const int64_t bt = rows > 1 ? table.stride(0) : width, bto = rows > 1 ? out.stride(0) : width;
    const c10::cuda::CUDAGuard guard(device);
    return unlocked(
        g_entries.reorder, dense<int32_t>(a[0], "parents", at::kInt, device, {B, K}),
        dense<int32_t>(a[1], "seqlens", at::kInt, device, {rows}), size_of(B, "the batch"),
        size_of(K, "the beams"), ptr<int32_t>(table), bt, size_of(width, "block_table"),
        int_of(a[5], "page_size"), ptr<int32_t>(pool),
        ptr<int32_t>(want(a[4], "free_count", at::kInt, device, {1})), pool.numel(),
        ptr<int32_t>(out), bto, dense<int32_t>(a[7], "seqlens_out", at::kInt, device, {rows}),
        dense<int32_t>(a[8], "copies", at::kInt, device, {rows, 3}),
        ptr<int32_t>(want(a[9], "free_count_out", at::kInt, device, {1})), err_of(a[10], device),
        stream_of(device));
  });
}

// copy_pages(copies, caches, err): caches a list or tuple of tensors
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 3)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& copies = tensor_of(a[0], "copies");
    const c10::Device device = device_of(copies, "copies");
    int32_t* list = dense<int32_t>(a[0], "copies", at::kInt, device, {-1, 3});
    const bool tuple = PyTuple_Check(a[1]);
    if (!tuple && !PyList_Check(a[1])) bad("caches", "must be a list or tuple of tensors");
    const Py_ssize_t count = tuple ? PyTuple_GET_SIZE(a[1]) : PyList_GET_SIZE(a[1]);
    std::vector<void*> at((size_t)count);
    int64_t st[3] = {16, 16, 16}, shape[4] = {1, 1, 1, 16}, size = 1;
    for (Py_ssize_t i = 0; i < count; ++i) {
      const at::Tensor& c =
          tensor_of(tuple ? PyTuple_GET_ITEM(a[1], i) : PyList_GET_ITEM(a[1], i), "caches");
      if (!c.is_cuda() || c.device() != device || c.dim() != 4 ||
          (c.size(3) > 1 && c.stride(3) != 1))
        bad("caches", "must be 4-d with a contiguous last axis, on the call's CUDA device");
      if (i == 0) {
        size = c.element_size();
        for (int x = 0; x < 4; ++x) shape[x] = c.size(x);
      }
      bool alike = (int64_t)c.element_size() == size;
      for (int x = 0; x < 4; ++x) alike = alike && c.size(x) == shape[x];
      for (int x = 2; x >= 0; --x) {
        // (the stride of an axis with one place does not matter)
        const int64_t s =
            shape[x] > 1 ? c.stride(x) * size : x == 2 ? shape[3] * size : st[x + 1] * shape[x + 1];
        alike = alike && (i == 0 || s == st[x]);
        st[x] = s;
      }
      if (!alike) bad("caches", "must have one shape, type and strides");
      at[(size_t)i] = c.data_ptr();
    }
    const c10::cuda::CUDAGuard guard(device);
    return unlocked(g_entries.copy, list, size_of(copies.size(0), "copies"), at.data(),
                    size_of(count, "caches"), st[0], st[1], st[2],
                    size_of(shape[3] * size, "the head size"), size_of(shape[2], "the heads"),
                    size_of(shape[1], "the page size"), shape[0], err_of(a[2], device),
                    stream_of(device));
  });
}

// fwd_cross(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, seqlens_k, key_mask,
//           scale, out, lse, workspace, err)
PyObject* fwd_cross(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 14)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& q = tensor_of(a[0], "q");
    const c10::Device device = device_of(q, "q");
    const at::ScalarType type = q.scalar_type();
    const int dtype = dtype_of(type);
    if (dtype < 0 || q.dim() != 3) bad("q", "must be a 3-d fp16 or bf16 tensor");
    const int64_t rows = q.size(0), hq = q.size(1), d = q.size(2);
    want(a[0], "q", type, device, {rows, hq, d});
    const auto& k = want(a[1], "k", type, device, {-1, -1, d});
    const int64_t keys = k.size(0), hkv = k.size(1);
    const auto& v = want(a[2], "v", type, device, {keys, hkv, d});
    const auto& cu_q = want(a[3], "cu_seqlens_q", at::kInt, device, {-1});
    const int64_t B = cu_q.numel() - 1;
    if (B < 0) bad("cu_seqlens_q", "must not be empty");
    const auto& cu_k = want(a[4], "cu_seqlens_k", at::kInt, device, {B + 1});
    const int32_t* lens =
        a[7] == Py_None ? nullptr : ptr<int32_t>(want(a[7], "seqlens_k", at::kInt, device, {B}));
    double scale = 0;
    if (a[9] == Py_None) {
      scale = 1.0 / std::sqrt((double)d);
    } else {
      scale = PyFloat_AsDouble(a[9]);
      if (scale == -1.0 && PyErr_Occurred()) throw PythonError();
    }
    float* lse = a[11] == Py_None ? nullptr : dense<float>(a[11], "lse", at::kFloat, device, {hq, rows});
    const auto& out = want(a[10], "out", type, device, {rows, hq, d});
    if (!out.is_contiguous()) bad("out", "must be contiguous");
    const c10::cuda::CUDAGuard guard(device);
    const int max_q = int_of(a[5], "max_seqlen_q");
    at::Tensor scratch;
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (a[12] != Py_None) {
      const at::Tensor& w = tensor_of(a[12], "workspace");
      if (!w.is_cuda() || w.device() != device || !w.is_contiguous())
        bad("workspace", "must be contiguous, on the call's CUDA device");
      ws = w.data_ptr();
      ws_bytes = (size_t)w.numel() * w.element_size();
    } else {
      ws_bytes = g_entries.cross_workspace(size_of(rows, "q"), max_q, size_of(hq, "q"),
                                           size_of(hkv, "k"), size_of(d, "q"));
      if (ws_bytes > 0) {
        scratch = at::empty({(int64_t)ws_bytes}, q.options().dtype(at::kByte));
        ws = scratch.data_ptr();
      }
    }
    return unlocked(
        g_entries.cross, q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(), k.stride(0),
        k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), ptr<int32_t>(cu_q), ptr<int32_t>(cu_k),
        lens, flags_of(a[8], "key_mask", device, {keys}), size_of(B, "the batch"),
        size_of(rows, "q"), size_of(keys, "k"), max_q,
        int_of(a[6], "max_seqlen_k"), size_of(hq, "q"), size_of(hkv, "k"), size_of(d, "q"),
        (float)scale, out.data_ptr(), lse, ws, ws_bytes, err_of(a[13], device), dtype, stream_of(device));
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction as_method() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef g_methods[] = {
    {"bind", as_method<bind>(), METH_FASTCALL, nullptr},
    {"bind_beam", as_method<bind_beam>(), METH_FASTCALL, nullptr},
    {"plan_step", as_method<plan_step>(), METH_FASTCALL, nullptr},
    {"release_pages", as_method<release_pages>(), METH_FASTCALL, nullptr},
    {"rotary_append_varlen", as_method<rotary_append_varlen>(), METH_FASTCALL, nullptr},
    {"fwd_varlen_e4m3", as_method<fwd_varlen_e4m3>(), METH_FASTCALL, nullptr},
    {"beam_select", as_method<beam_select>(), METH_FASTCALL, nullptr},
    {"beam_reorder", as_method<beam_reorder>(), METH_FASTCALL, nullptr},
    {"copy_pages", as_method<copy_pages>(), METH_FASTCALL, nullptr},
    {"fwd_cross", as_method<fwd_cross>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&g_module); }
