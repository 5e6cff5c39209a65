// Rotary embedding of a ragged batch's new tokens by positions with one or
// several axes, and the write of their k and v into the paged cache's slots,
// in 16 bits or as e4m3 (sm_103a): the step between the projections and
// pa_fwd_varlen_unified / pa_fwd_varlen_e4m3, whose chunks must already be in
// the cache (vLLM #6052 "Unify the kernel used in flash attention backend";
// the separate cache write of vLLM #3010 "Introduce flash-attn"; the fused
// rotary embedding named on flash-attention #824).
//
// Mathematics.  Pair p of a token's features turns by the angle of the
// token's position on the pair's axis a(p): with c = cos[pos_a(p)][p] and s
// alike, (x1, x2) -> (x1 c - x2 s, x1 s + x2 c), in fp32.  q and a 16-bit
// cache round that once to their type; an e4m3 cache rounds the fp32 quotient
// x / scale once, saturating at +-448.  16 fp32 divisions a thread and row would
// be half of the kernel's instructions: products by both ends of an interval
// around 1 / scale show nearly always what the quotient rounds to (Divisor, below;
// 8192 tokens of 32/8 heads 36.8 us, with divisions alone 38.5).
//
// Bound: memory; every byte of q, k and v is read once and of q_out and the
// slots written once.  A thread owns 16 features of a head row -- features
// [8u, 8u + 8) and their partners half a rotation further on, or 16 adjacent
// ones for even/odd pairs -- so that a rotation needs no other thread, every
// access is 16 bytes wide (8 for e4m3 stores) and the threads of a row cover
// whole 64- or 128-byte runs.  The angles of a thread's 8 pairs depend on the
// token alone: they are loaded once and serve every head row the thread takes.
#include <cuda_fp8.h>

#include <algorithm>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
int set_error(int code, const char* fmt, ...);

namespace {

constexpr int kMaxAxes = 4;
constexpr int kMaxPairs = 64;
constexpr int kThreads = 256;
// Head rows a thread has in flight where it takes several of a tensor, and
// resident blocks of an SM: 2 and 4 (64 registers) run 8192 tokens of 32/8 heads
// in 37 us; 1 and 4 take 39, 4 and 2 take 46, 3 and 3 take 42, 2 and 5 spill and
// take 46.  Rows by way of shared memory, four or six of them ahead, took 1.5 us
// more than these.
constexpr int kBatch = 2, kBlocks = 4;
constexpr int kWarpsWanted = 152 * 64;  // two rounds of the GPU's warps

struct RotAppendParams {
  const void *q, *k, *v;
  void* q_out;
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, qo_st, qo_sh;
  void *k_cache, *v_cache;
  int64_t kc_sb, kc_st, kc_sh, vc_sb, vc_st, vc_sh;
  const float *k_scale, *v_scale;
  const int64_t* slots;
  const int32_t* positions;
  int64_t pos_stride;
  const void *cos, *sin;
  int64_t num_slots;
  int32_t* err;
  int T, Hq, Hkv, page_log2;  // Hq: 0 without q
  int n_axes, rot_len, rot, interleaved, table_f32, parts, roles;
  unsigned char axis[kMaxPairs];
  uint32_t unit_axes[kMaxPairs / 8];  // byte a: which of the unit's 8 pairs axis a turns
};

// As load16, without the promise that nothing writes there while the kernel
// runs: q_out may be q.
__device__ __forceinline__ uint4 load16_rw(const void* src) {
  uint4 x;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(src));
  return x;
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float* x) {
  using E = Elem<T>;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = E::to_f2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float* x) {
  using E = Elem<T>;
  return make_uint4(E::from_f2(x[0], x[1]), E::from_f2(x[2], x[3]), E::from_f2(x[4], x[5]),
                    E::from_f2(x[6], x[7]));
}
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// What a head's values are divided by, and the ends of an interval that holds
// 1 / scale: its fp32 reciprocal, off by at most 2^-24 of itself, moved by 5 and
// 6 times that.  Rounding the end and x times it adds 2^-24 each, rounding x /
// scale to fp32 another, so that the two products enclose the fp32 quotient;
// conversion to e4m3 is monotonic, so where both convert alike the quotient
// converts to the same.  Quotients next to a midpoint of two e4m3 values, about
// one of 2^17, are computed, and all of those by a scale whose reciprocal may
// not be a normal number: its ends never convert alike (0 x 0 and 0 x inf
// neither), but for NaN.
struct Divisor {
  float scale = 1.f, lo = 1.f, hi = 1.f;
  __device__ __forceinline__ explicit Divisor(const float* s) {
    if (s == nullptr) return;
    scale = __ldg(s);
    const float r = __frcp_rn(scale);
    const bool normal = fabsf(scale) >= 0x1p-120f && fabsf(scale) <= 0x1p120f;
    lo = normal ? r * (1.f - 5 * 0x1p-24f) : 0.f;
    hi = normal ? r * (1.f + 6 * 0x1p-24f) : __int_as_float(0x7f800000);
  }
};
__device__ __forceinline__ uint32_t e4m3x4(const float* x, float by) {
  return e4m3x2(x[0] * by, x[1] * by) | (e4m3x2(x[2] * by, x[3] * by) << 16);
}
// e4m3(x / scale) of the 16 values of a thread, 8 in `a` and 8 in `b`.
__device__ __forceinline__ void quotients_e4m3(const float (&a)[8], const float (&b)[8],
                                               const Divisor& d, uint32_t (&y)[4]) {
  uint32_t apart = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* x = (i < 2 ? a : b) + (i & 1) * 4;
    y[i] = e4m3x4(x, d.lo);
    apart |= y[i] ^ e4m3x4(x, d.hi);
  }
  if (apart == 0) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* x = (i < 2 ? a : b) + (i & 1) * 4;
    y[i] = e4m3x2(__fdiv_rn(x[0], d.scale), __fdiv_rn(x[1], d.scale)) |
           (e4m3x2(__fdiv_rn(x[2], d.scale), __fdiv_rn(x[3], d.scale)) << 16);
  }
}

template <typename T>
__device__ __forceinline__ float table_at(const void* t, int64_t i, bool f32) {
  return f32 ? __ldg(reinterpret_cast<const float*>(t) + i)
             : static_cast<float>(reinterpret_cast<const T*>(t)[i]);
}

// Where the token's k and v go: an element offset in either cache, or false
// for a token without a slot.
__device__ __forceinline__ bool slot_of(const RotAppendParams& p, int t, bool tell, int64_t* k_off,
                                        int64_t* v_off) {
  const int64_t slot = __ldg(p.slots + t);
  if (slot < 0) return false;
  if (slot >= p.num_slots) {
    if (tell)
      report(p.err, PA_DEVERR_PAGE_OOB, t,
             (int)min(slot >> p.page_log2, (int64_t)0x7fffffff));
    return false;
  }
  const int64_t page = slot >> p.page_log2, row = slot & ((1 << p.page_log2) - 1);
  *k_off = page * p.kc_sb + row * p.kc_st;
  *v_off = page * p.vc_sb + row * p.vc_st;
  return true;
}

// False (and a report) if a position of the token lies outside the tables.
__device__ __forceinline__ bool positions_of(const RotAppendParams& p, int t, bool tell, int* pos) {
  bool ok = true;
#pragma unroll
  for (int a = 0; a < kMaxAxes; ++a) {
    pos[a] = 0;
    if (a >= p.n_axes) continue;
    pos[a] = __ldg(p.positions + a * p.pos_stride + t);
    if (pos[a] < 0 || pos[a] >= p.rot_len) {
      if (ok && tell) report(p.err, PA_DEVERR_LENGTH, t, pos[a]);
      ok = false;
    }
  }
  return ok;
}

__device__ __forceinline__ int pick(const int* pos, int a) {
  return a == 0 ? pos[0] : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3];
}

// The cosines or sines of a unit's 8 pairs from row `at` of a table.
template <typename T>
__device__ __forceinline__ void table8(const void* t, int64_t at, int f32, float (&x)[8]) {
  if (f32) {
    const float* src = reinterpret_cast<const float*>(t) + at;
    const uint4 lo = load16(src), hi = load16(src + 4);
    x[0] = __uint_as_float(lo.x); x[1] = __uint_as_float(lo.y);
    x[2] = __uint_as_float(lo.z); x[3] = __uint_as_float(lo.w);
    x[4] = __uint_as_float(hi.x); x[5] = __uint_as_float(hi.y);
    x[6] = __uint_as_float(hi.z); x[7] = __uint_as_float(hi.w);
  } else {
    unpack8<T>(load16(reinterpret_cast<const T*>(t) + at), x);
  }
}

// Each warp takes part `part` of `parts` of one token's head rows, 32 / (D / 16)
// rows at a time: first k and v, then q.
// BATCH rows of a thread are in flight.
template <int D, typename T, bool E4M3, int BATCH>
__global__ void __launch_bounds__(kThreads, kBlocks) rotary_append_kernel(
    const __grid_constant__ RotAppendParams p) {
  constexpr int kPerRow = D / 16;           // threads of a head row
  constexpr int kRows = 32 / kPerRow;       // head rows of a warp at a time
  const int lane = threadIdx.x & 31;
  const long long w = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int shares = p.parts * p.roles;
  if (w >= (long long)p.T * shares) return;
  const int t = shares == 1 ? (int)w : (int)(w / shares);
  const int share = shares == 1 ? 0 : (int)(w % shares);
  const int role = p.roles == 1 ? -1 : share % 3, part = share / p.roles;  // 0: k, 1: v, 2: q
  const int u = lane % kPerRow;
  const int units = p.rot >> 4;             // units that turn
  int lo, hi;                               // the unit's two runs of 8 features
  if (!p.interleaved && u < units) {
    lo = 8 * u;
    hi = (p.rot >> 1) + 8 * u;
  } else {
    lo = 16 * u;
    hi = 16 * u + 8;
  }
  const bool tell = share == 0 && lane == 0;
  int64_t k_off = 0, v_off = 0;
  const bool live = role != 2 && slot_of(p, t, tell, &k_off, &v_off);
  float c[8], s[8];
  bool turns = false;
  if (p.cos != nullptr && role != 1) {
    int pos[kMaxAxes];
    turns = positions_of(p, t, tell, pos) && u < units;
    if (turns) {
      // one row of the tables an axis that the unit's pairs use
      const uint32_t masks = p.unit_axes[u];
      const int half = p.rot >> 1;
      table8<T>(p.cos, (int64_t)pos[0] * half + 8 * u, p.table_f32, c);
      table8<T>(p.sin, (int64_t)pos[0] * half + 8 * u, p.table_f32, s);
#pragma unroll
      for (int a = 1; a < kMaxAxes; ++a) {
        if (a >= p.n_axes) break;
        const uint32_t mask = (masks >> (8 * a)) & 0xffu;
        float ca[8], sa[8];
        table8<T>(p.cos, (int64_t)pos[a] * half + 8 * u, p.table_f32, ca);
        table8<T>(p.sin, (int64_t)pos[a] * half + 8 * u, p.table_f32, sa);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          c[i] = (mask >> i) & 1 ? ca[i] : c[i];
          s[i] = (mask >> i) & 1 ? sa[i] : s[i];
        }
      }
    }
  }
  auto rotate = [&](float (&a)[8], float (&b)[8]) {
    if (!p.interleaved) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = fmaf(a[e], c[e], -(b[e] * s[e]));
        b[e] = fmaf(a[e], s[e], b[e] * c[e]);
        a[e] = y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float y = fmaf(a[e], c[e / 2], -(a[e + 1] * s[e / 2]));
        a[e + 1] = fmaf(a[e], s[e / 2], a[e + 1] * c[e / 2]);
        a[e] = y;
        const float z = fmaf(b[e], c[4 + e / 2], -(b[e + 1] * s[4 + e / 2]));
        b[e + 1] = fmaf(b[e], s[4 + e / 2], b[e + 1] * c[4 + e / 2]);
        b[e] = z;
      }
    }
  };
  const int first = part * kRows + lane / kPerRow, step = kRows * p.parts;
  // The head rows first, first + step, ... of one tensor, BATCH of them in
  // flight: loads without a condition (a row behind the last is read as the
  // thread's own first of them: another's may be written already), or they would
  // wait for one another.  `put` stores row r.
  auto rows = [&](const T* src, int64_t sh, int n, auto&& put) {
#pragma unroll 1
    for (int r0 = first; r0 < n; r0 += step * BATCH) {
      uint4 x_lo[BATCH], x_hi[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const T* row = src + (r0 + i * step < n ? r0 + i * step : r0) * sh;
        x_lo[i] = load16_rw(row + lo);
        x_hi[i] = load16_rw(row + hi);
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
        if (r0 + i * step < n) put(r0 + i * step, x_lo[i], x_hi[i]);
    }
  };
  auto store = [&](T* dst, const uint4& x_lo, const uint4& x_hi, bool turn) {
    uint4 y_lo = x_lo, y_hi = x_hi;
    if (turn) {
      float a[8], b[8];
      unpack8<T>(x_lo, a);
      unpack8<T>(x_hi, b);
      rotate(a, b);
      y_lo = pack8<T>(a);
      y_hi = pack8<T>(b);
    }
    *reinterpret_cast<uint4*>(dst + lo) = y_lo;
    *reinterpret_cast<uint4*>(dst + hi) = y_hi;
  };
  if (live) {
#pragma unroll 1
    for (int kv = 0; kv < 2; ++kv) {
      if (role >= 0 && role != kv) continue;
      const bool turn = kv == 0 && turns;
      const T* src = kv == 0 ? reinterpret_cast<const T*>(p.k) + t * p.k_st
                             : reinterpret_cast<const T*>(p.v) + t * p.v_st;
      const int64_t off = kv == 0 ? k_off : v_off, sh = kv == 0 ? p.kc_sh : p.vc_sh;
      void* cache = kv == 0 ? p.k_cache : p.v_cache;
      const float* scales = kv == 0 ? p.k_scale : p.v_scale;
      rows(src, kv == 0 ? p.k_sh : p.v_sh, p.Hkv, [&](int h, const uint4& x_lo, const uint4& x_hi) {
        if constexpr (E4M3) {
          const Divisor by(scales != nullptr ? scales + h : nullptr);
          float a[8], b[8];
          unpack8<T>(x_lo, a);
          unpack8<T>(x_hi, b);
          if (turn) rotate(a, b);
          uint32_t y[4];
          quotients_e4m3(a, b, by, y);
          uint8_t* dst = reinterpret_cast<uint8_t*>(cache) + off + h * sh;
          *reinterpret_cast<uint2*>(dst + lo) = make_uint2(y[0], y[1]);
          *reinterpret_cast<uint2*>(dst + hi) = make_uint2(y[2], y[3]);
        } else {
          store(reinterpret_cast<T*>(cache) + off + h * sh, x_lo, x_hi, turn);
        }
      });
    }
  }
  if (role == 0 || role == 1) return;
  rows(reinterpret_cast<const T*>(p.q) + t * p.q_st, p.q_sh, p.Hq,
       [&](int h, const uint4& x_lo, const uint4& x_hi) {
         store(reinterpret_cast<T*>(p.q_out) + t * p.qo_st + h * p.qo_sh, x_lo, x_hi, turns);
       });
}

// Rotations whose width is no multiple of 16 features, and tables that are not
// 16-byte aligned: a thread takes one pair (or two features that do not turn) of one head row.
template <int D, typename T, bool E4M3>
__global__ void __launch_bounds__(kThreads) rotary_append_pairs_kernel(const __grid_constant__
                                                                           RotAppendParams p) {
  const int rows = p.Hq + 2 * p.Hkv, turned_rows = p.Hq + p.Hkv;
  const long long all = (long long)p.T * rows * (D / 2);
  const long long stride = (long long)gridDim.x * kThreads;
  for (long long x = (long long)blockIdx.x * kThreads + threadIdx.x; x < all; x += stride) {
    const int f = (int)(x % (D / 2));
    const int r = (int)((x / (D / 2)) % rows);
    const int t = (int)(x / ((long long)rows * (D / 2)));
    const bool tell = r == 0 && f == 0;
    const bool in = f < p.rot / 2;
    const int i1 = !in || p.interleaved ? 2 * f : f;
    const int i2 = !in || p.interleaved ? 2 * f + 1 : f + p.rot / 2;
    const T* src;
    if (r < p.Hq)
      src = reinterpret_cast<const T*>(p.q) + t * p.q_st + r * p.q_sh;
    else if (r < turned_rows)
      src = reinterpret_cast<const T*>(p.k) + t * p.k_st + (r - p.Hq) * p.k_sh;
    else
      src = reinterpret_cast<const T*>(p.v) + t * p.v_st + (r - turned_rows) * p.v_sh;
    float y1 = static_cast<float>(src[i1]), y2 = static_cast<float>(src[i2]);
    int pos[kMaxAxes];
    const bool ok = positions_of(p, t, tell, pos);
    if (ok && in && r < turned_rows) {
      const int64_t at = (int64_t)pick(pos, p.axis[f]) * (p.rot / 2) + f;
      const float c = table_at<T>(p.cos, at, p.table_f32), s = table_at<T>(p.sin, at, p.table_f32);
      const float z = fmaf(y1, c, -(y2 * s));
      y2 = fmaf(y1, s, y2 * c);
      y1 = z;
    }
    int64_t k_off = 0, v_off = 0;
    const bool live = slot_of(p, t, tell, &k_off, &v_off);
    if (r < p.Hq) {
      T* dst = reinterpret_cast<T*>(p.q_out) + t * p.qo_st + r * p.qo_sh;
      dst[i1] = Elem<T>::from_f(y1);
      dst[i2] = Elem<T>::from_f(y2);
      continue;
    }
    if (!live) continue;
    const bool is_k = r < turned_rows;
    const int h = r - (is_k ? p.Hq : turned_rows);
    const int64_t off = is_k ? k_off + h * p.kc_sh : v_off + h * p.vc_sh;
    if constexpr (E4M3) {
      const float* scales = is_k ? p.k_scale : p.v_scale;
      const float by = scales != nullptr ? __ldg(scales + h) : 1.f;
      const uint32_t u = e4m3x2(__fdiv_rn(y1, by), __fdiv_rn(y2, by));
      uint8_t* dst = reinterpret_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) + off;
      dst[i1] = (uint8_t)(u & 0xff);
      dst[i2] = (uint8_t)(u >> 8);
    } else {
      T* dst = reinterpret_cast<T*>(is_k ? p.k_cache : p.v_cache) + off;
      dst[i1] = Elem<T>::from_f(y1);
      dst[i2] = Elem<T>::from_f(y2);
    }
  }
}

template <int D, typename T, bool E4M3>
cudaError_t launch(RotAppendParams& p, cudaStream_t st) {
  const int rows = p.Hq + 2 * p.Hkv;
  const uintptr_t tables = reinterpret_cast<uintptr_t>(p.cos) | reinterpret_cast<uintptr_t>(p.sin);
  if (p.cos != nullptr && (p.rot % 16 != 0 || (tables & 15u) != 0)) {
    const long long blocks = ((long long)p.T * rows * (D / 2) + kThreads - 1) / kThreads;
    rotary_append_pairs_kernel<D, T, E4M3>
        <<<(unsigned)std::min<long long>(blocks, 152 * 32), kThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  // Warps of a token: one where the tokens alone fill the GPU (the angles are
  // then loaded once a token; two warps a token took 42 us instead of 35 for 8192 tokens of
  // 32/8 heads), for fewer tokens more of them, and where one round of the GPU's
  // warps holds them one for every set of rows of q, of k and of v (64 tokens:
  // 3.5 -> 2.5 us; 1601 tokens of 12/12 heads, two rounds: 5.4 -> 7.3 us).
  const int per = 32 / (D / 16);
  const int most = (std::max(p.Hq, p.Hkv) + per - 1) / per;
  const long long want = kWarpsWanted;
  p.parts = (int)std::max<long long>(1, std::min<long long>(most, want / p.T));
  p.roles = p.parts == most && (long long)p.T * p.parts * 6 <= want ? 3 : 1;
  const long long blocks = ((long long)p.T * p.parts * p.roles * 32 + kThreads - 1) / kThreads;
  // A thread that has one row of each tensor loads one at a time: 8 % less for 64
  // tokens (now 2.4 us), 9 % less for 1601 tokens of 12/12 heads (5.2 us).
  if (p.parts == most)
    rotary_append_kernel<D, T, E4M3, 1><<<(unsigned)blocks, kThreads, 0, st>>>(p);
  else
    rotary_append_kernel<D, T, E4M3, kBatch><<<(unsigned)blocks, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <int D, typename T>
cudaError_t launch_cache(RotAppendParams& p, bool e4m3, cudaStream_t st) {
  return e4m3 ? launch<D, T, true>(p, st) : launch<D, T, false>(p, st);
}

bool aligned16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }

// Rows of 16-bit elements that are read or written 16 bytes at a time.
int check_rows(const void* ptr, int64_t st, int64_t sh, const char* name) {
  if (ptr == nullptr) return set_error(PA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(ptr) || st <= 0 || sh <= 0 || st % 8 != 0 || sh % 8 != 0)
    return set_error(PA_ERR_INVALID_ARG,
                     "%s must be 16-byte aligned with positive strides in multiples of 8 elements",
                     name);
  return PA_OK;
}

int check_slots(const pa_tensor4& t, bool e4m3, const char* name) {
  const int64_t m = e4m3 ? 16 : 8;
  if (t.ptr == nullptr) return set_error(PA_ERR_INVALID_ARG, "%s.ptr is NULL", name);
  if (!aligned16(t.ptr) || t.stride_b <= 0 || t.stride_t <= 0 || t.stride_h <= 0 ||
      t.stride_b % m != 0 || t.stride_t % m != 0 || t.stride_h % m != 0)
    return set_error(PA_ERR_INVALID_ARG,
                     "%s must be 16-byte aligned with positive strides in multiples of 16 bytes",
                     name);
  return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

PA_API int pa_rotary_append_varlen(
    const void* q, int64_t q_st, int64_t q_sh, const void* k, int64_t k_st, int64_t k_sh,
    const void* v, int64_t v_st, int64_t v_sh, void* q_out, int64_t qo_st, int64_t qo_sh,
    pa_tensor4 k_cache, pa_tensor4 v_cache, const float* k_scale, const float* v_scale,
    const int64_t* slot_mapping, int page_size, int64_t num_pages, const int32_t* positions,
    int64_t pos_stride, int n_axes, const uint8_t* pair_axis, const void* rotary_cos,
    const void* rotary_sin, int rotary_len, int rotary_dim, int rotary_interleaved,
    int rotary_dtype, int T, int Hq, int Hkv, int D, int dtype, int cache_dtype,
    int32_t* err_word, pa_stream_t stream) {
  if (dtype != PA_F16 && dtype != PA_BF16) return set_error(PA_ERR_UNSUPPORTED, "dtype %d", dtype);
  if (cache_dtype != dtype && cache_dtype != PA_E4M3)
    return set_error(PA_ERR_UNSUPPORTED, "a cache holds the dtype of k and v or PA_E4M3");
  const bool e4m3 = cache_dtype == PA_E4M3;
  if (D != 64 && D != 128) return set_error(PA_ERR_UNSUPPORTED, "head_dim %d (64 or 128)", D);
  if (T < 0) return set_error(PA_ERR_INVALID_ARG, "negative T");
  if (Hkv < 1 || (q != nullptr && Hq < 1))
    return set_error(PA_ERR_INVALID_ARG, "head counts must be >= 1");
  if (T == 0) return PA_OK;
  int rc = 0;
  if ((rc = check_slots(k_cache, e4m3, "k_cache")) || (rc = check_slots(v_cache, e4m3, "v_cache")) ||
      (rc = check_rows(k, k_st, k_sh, "k")) || (rc = check_rows(v, v_st, v_sh, "v")))
    return rc;
  if (q != nullptr && ((rc = check_rows(q, q_st, q_sh, "q")) ||
                       (rc = check_rows(q_out, qo_st, qo_sh, "q_out"))))
    return rc;
  if (slot_mapping == nullptr) return set_error(PA_ERR_INVALID_ARG, "slot_mapping is NULL");
  if (num_pages < 1) return set_error(PA_ERR_INVALID_ARG, "num_pages must be >= 1");
  RotAppendParams p{};
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) p.page_log2 = s;
  if (p.page_log2 == 0)
    return set_error(PA_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
  if (rotary_cos != nullptr) {
    if (rotary_sin == nullptr || positions == nullptr)
      return set_error(PA_ERR_INVALID_ARG, "a rotation needs rotary_sin and positions");
    if (rotary_dim < 2 || rotary_dim > D || rotary_dim % 2 != 0 || rotary_len < 1)
      return set_error(PA_ERR_INVALID_ARG,
                       "rotary_dim must be even in [2, D] and rotary_len >= 1");
    if (rotary_dtype != dtype && rotary_dtype != PA_F32)
      return set_error(PA_ERR_UNSUPPORTED, "the rotary tables hold the dtype of q or PA_F32");
    if (n_axes < 1 || n_axes > kMaxAxes || (n_axes > 1 && pos_stride < T))
      return set_error(PA_ERR_INVALID_ARG, "n_axes must be 1 to %d, with pos_stride >= T", kMaxAxes);
    for (int i = 0; i < rotary_dim / 2; ++i) {
      p.axis[i] = pair_axis != nullptr ? pair_axis[i] : 0;
      if (p.axis[i] >= n_axes)
        return set_error(PA_ERR_INVALID_ARG, "pair_axis[%d] = %d names no axis", i, (int)p.axis[i]);
      p.unit_axes[i / 8] |= 1u << (8 * p.axis[i] + i % 8);
    }
    p.cos = rotary_cos;
    p.sin = rotary_sin;
    p.positions = positions;
    p.pos_stride = pos_stride;
    p.n_axes = n_axes;
    p.rot_len = rotary_len;
    p.rot = rotary_dim;
    p.interleaved = rotary_interleaved ? 1 : 0;
    p.table_f32 = rotary_dtype == PA_F32 ? 1 : 0;
  }
  p.q = q; p.q_st = q_st; p.q_sh = q_sh;
  p.k = k; p.k_st = k_st; p.k_sh = k_sh;
  p.v = v; p.v_st = v_st; p.v_sh = v_sh;
  p.q_out = q_out; p.qo_st = qo_st; p.qo_sh = qo_sh;
  p.k_cache = k_cache.ptr;
  p.v_cache = v_cache.ptr;
  p.kc_sb = k_cache.stride_b; p.kc_st = k_cache.stride_t; p.kc_sh = k_cache.stride_h;
  p.vc_sb = v_cache.stride_b; p.vc_st = v_cache.stride_t; p.vc_sh = v_cache.stride_h;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.slots = slot_mapping;
  p.num_slots = num_pages << p.page_log2;
  p.T = T;
  p.Hq = q != nullptr ? Hq : 0;
  p.Hkv = Hkv;
  p.err = err_word;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == PA_F16)
    e = D == 128 ? launch_cache<128, __half>(p, e4m3, st) : launch_cache<64, __half>(p, e4m3, st);
  else
    e = D == 128 ? launch_cache<128, __nv_bfloat16>(p, e4m3, st)
                 : launch_cache<64, __nv_bfloat16>(p, e4m3, st);
  if (e != cudaSuccess)
    return set_error(PA_ERR_CUDA, "rotary append launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

}  // extern "C"
