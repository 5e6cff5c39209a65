// A beam search's selection over beams and vocabulary (sm_103a): from the logits
// of every beam the best continuations of each request (pa_beam_select).
//
// Mathematics.  Beam k of a request has the score s_k and the logits x_k[v]:
//   lse_k = ln sum_v exp(x_k[v]),   score(k, v) = s_k + (x_k[v] - lse_k),
// and the N largest scores over all (k, v) are wanted, in order, the lowest
// k * V + v first among equal ones.  exp is taken as 2^(x log2(e) - n) against
// a whole number n, so that sums under different references are brought
// together by exact powers of two; log2(e) is a sum of two fp32 values, which
// leaves one rounding of the exponent.  (Where the largest logit is beyond 2^29 an
// fp32 n is too coarse: see Reference.)  The exponentials, and the 64 of a lane's step,
// are fp32: lse is good to 2^-17, and so is the order of two beams' candidates.  Nothing
// behind them adds to that, whatever the row's length: what a lane's steps add up to, the
// sums of a row's parts and its logarithm (ln f = 2 atanh((f - 1) / (f + 1))) are in pairs
// of fp32 values, the candidates' scores in 64 bits, so the order within a beam is that of
// 64 bits.  (FP64 is slow here: log() of a double took 5500 cycles, the pairs take 700.)
//
// One pass over the logits, 4 KB of a warp on their way while it computes with the
// 4 KB before.  A lane finds the maximum of its elements, then their sum.  Only the
// maxima are kept (one of 32 or more elements, in shared memory).  The N largest
// elements lie in blocks whose maximum is among the N largest maxima, so a bound
// found from the maxima leaves a few dozen blocks, whose elements are read once more
// (from L2) and ranked.  Where more elements than fit pass the bound (many equal logits), the
// N best are found one after the other.
//
// A cluster of up to 16 CTAs per request: the beams of a request must be
// compared with one another, and over distributed shared memory that takes two
// barriers, no scratch memory and no second launch.
//
// Ties.  Equal rows are equal candidates, but where their addresses differ modulo 16
// bytes they are cut into other vectors and their sums are added up in another order.
// So a row has a code, the sum of its elements' bits, which does not depend on the
// order: rows of one code whose lse agree within what the sums may be off have the lse
// of the first.
//
// Measured: 64 requests of 8 beams, 128000 bf16 logits: 36.5 us, 20 of them the pass
// (6.5 TB/s), the others start, sums, bound, candidates and the join, as in 8.2 us for
// one request of 4 beams of 32000.  16 of 5 beams of an odd number of logits 12.8 (12.1
// without codes and pairs).  More than 32 candidates where a CTA has one unit of a row:
// half of the parts are empty, nothing bounds the candidates, and all elements are
// compared N times (32 beams of 32000 bf16 logits, one request: N = 32 36 us, 33 5200 us,
// 64 10060 us).
#include <cooperative_groups.h>

#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kThreads = 512;      // (two CTAs of 256 an SM: 26.7 us for 21.8, 8 requests of 16 beams)
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 1;
constexpr int kVecs = 8;           // 16-byte vectors of a lane in a step
constexpr int kStepVecs = 32 * kVecs;
constexpr int kMaxBeams = 32;
constexpr int kMaxOut = 64;
constexpr int kParts = 64;         // of the block maxima: the N-th largest of their maxima is the bound
constexpr int kMaxCandidates = 1024;
constexpr int kMaxCluster = kClusterLimit;
constexpr int kMaxUnits = 64;      // of a CTA
constexpr uint32_t kAll = 0xffffffffu;

constexpr float kLog2eHi = 1.44269502163f;  // log2(e) to fp32, and what is missing
constexpr float kLog2eLo = 1.92596299e-8f;
constexpr double kLn2d = 0.69314718055994530942;

struct SelectParams {
  const void* logits;
  int64_t stride_b, stride_k;
  const float* scores;
  const uint8_t* finished;
  int end_token;
  int B, K, V, N;
  int steps;      // steps of kStepVecs vectors in a unit
  int row_units;  // units of a row
  float* scores_out;
  int32_t* parents;
  int32_t* tokens;
  uint8_t* finished_out;
  int32_t* err;
};

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 16 bytes of logits.
template <typename T>
struct Logits {
  static constexpr int kPer = 16 / sizeof(T);
  static __device__ __forceinline__ uint4 none() {  // -inf everywhere
    const uint32_t u = std::is_same<T, float>::value    ? 0xff800000u
                       : std::is_same<T, __half>::value ? 0xfc00fc00u
                                                        : 0xff80ff80u;
    return make_uint4(u, u, u, u);
  }
  static __device__ __forceinline__ void expand(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (std::is_same<T, float>::value) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = Elem<T>::to_f2(w[i]);
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
      }
    }
  }
  // The largest of a lane's vectors (NaN does not count).
  static __device__ __forceinline__ float largest(const uint4 (&v)[kVecs]) {
    if constexpr (std::is_same<T, float>::value) {
      float m = neg_inf();
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(v[j].x), __uint_as_float(v[j].y)),
                           fmaxf(__uint_as_float(v[j].z), __uint_as_float(v[j].w))));
      return m;
    } else {
      using T2 = typename Elem<T>::T2;
      auto as = [](uint32_t u) { return *reinterpret_cast<T2*>(&u); };
      T2 m = as(v[0].x);
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        m = __hmax2(m, __hmax2(__hmax2(as(v[j].x), as(v[j].y)), __hmax2(as(v[j].z), as(v[j].w))));
      const float2 f = Elem<T>::to_f2(*reinterpret_cast<uint32_t*>(&m));
      return fmaxf(f.x, f.y);
    }
  }
  // The sum of the values' bits but for their signs (+0 and -0 are equal), on top of c.
  // (Of fp32 values it counts modulo 2^31.)
  static __device__ __forceinline__ uint32_t code(const uint4& v, uint32_t c) {
    if constexpr (std::is_same<T, float>::value) return c + v.x + v.y + v.z + v.w;
    else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) c = __dp2a_lo(w[i] & 0x7fff7fffu, 0x101u, c);
      return c;
    }
  }
  static __device__ __forceinline__ uint32_t bits(const T* p) {
    if constexpr (std::is_same<T, float>::value) return __float_as_uint(*p);
    else return *reinterpret_cast<const uint16_t*>(p);
  }
  static constexpr uint32_t kCode = std::is_same<T, float>::value ? 0x7fffffffu : 0xffffffffu;
  static __device__ __forceinline__ float one(const T* p) { return (float)*p; }
  // A first word whose first value is *p, the others -inf.
  static __device__ __forceinline__ uint32_t alone(const T* p) {
    if constexpr (std::is_same<T, float>::value) return __float_as_uint(*p);
    else return (none().x & 0xffff0000u) | bits(p);
  }
};

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}

// A sum in a pair of fp32 values (the second is what the first lacks), times
// 4^h (h the half of a whole number), or e^h where |h| >= kFar.
struct Sum {
  float h, hi, lo;
};
constexpr float kFar = 0x1p29f;
constexpr float kNothing = -3.402823466e38f;  // h where there is nothing but -inf
// 4^d for a half of a whole number d <= 0 (0 below the normal range).
__device__ __forceinline__ float pow4(float d) {
  return d < -63.f ? 0.f : __int_as_float((127 + (int)(2.f * d)) << 23);
}
// What the exponentials of values whose largest is `top` are taken against:
// x stands for 2^(x hi + x lo - minus).  Nearer to 0 than kFar that is e^x / 4^h.
// Beyond it h is top itself (behind those of smaller values, 0.72 x), and for
// e^(x - top) stands 4^(x - top), or 2^((x - top) 2^-20) where 2 x might not be
// finite: 1 at top, and no more than 2^-64 at any other x, which lies 32 below at
// least, where e^-32 adds 2^-22 to a sum even as one of 2^24.  (lo: -inf times 0
// would be NaN.)
struct Reference {
  float h, hi, lo, minus;
};
template <typename T>
__device__ __forceinline__ Reference reference_of(float top) {
  const float n = rintf(top * kLog2eHi);
  if constexpr (std::is_same<T, __half>::value) {  // (finite ones lie above -2^17)
    const float m = fmaxf(n, -0x1p20f);
    return {m == n ? 0.5f * m : kNothing, kLog2eHi, kLog2eLo, m};
  } else {
    const float t = fmaxf(top, kNothing);
    if (fabsf(t) < kFar) return {0.5f * n, kLog2eHi, kLog2eLo, n};
    const float by = fabsf(t) < 0x1p60f ? 2.f : 0x1p-20f;
    return {t, by, 0x1p-126f, t * by};
  }
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, o));
  return x;
}
// Over the warp, the same in every lane (x + y and what it lacks do not depend
// on their order).
__device__ __noinline__ Sum warp_total(Sum s) {
  const float h = warp_max(s.h), f = pow4(s.h - h);
  float hi = s.hi * f, lo = s.lo * f;
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(kAll, hi, o), z = __shfl_xor_sync(kAll, lo, o);
    const float t = hi + y, u = t - hi;
    const float e = ((hi - (t - u)) + (y - u)) + (lo + z);
    hi = t + e;
    lo = e - (hi - t);
  }
  return {h, hi, lo};
}
// ln(s), s positive and finite.
__device__ __forceinline__ double ln_of(const Sum& s) {
  // s = 2^e f with f in [0.7, 1.42)
  const int bits = __float_as_int(s.hi);
  const int e = (bits - 0x3f350000) >> 23;
  const float down = __int_as_float((127 - e) << 23);
  const float f = s.hi * down, g = s.lo * down;
  const float num = f - 1.f, den = f + 1.f;  // num is exact
  const float den_lo = (1.f - (den - f)) + g;
  const float q = __fdividef(num, den);  // (what it lacks is in r)
  const float r = __fdividef(fmaf(-q, den, num) + (g - q * den_lo), den);
  const float z = q * q;
  const float t = fmaf(fmaf(fmaf(fmaf(z, 1.f / 11, 1.f / 9), z, 1.f / 7), z, 1.f / 5), z, 1.f / 3);
  const bool far = fabsf(s.h) >= kFar;
  const double whole = far ? (double)e : 2.0 * (double)s.h + e;
  const double ln = whole * kLn2d + (2.0 * (double)q + (double)(2.f * (r + q * z * t)));
  return far ? (double)s.h + ln : ln;  // (rounded to h's size once)
}

// Larger is better; a score's order as a whole number (+0 and -0 alike).
__device__ __forceinline__ long long order_of(double s) {
  const long long b = __double_as_longlong(s + 0.0);
  return b ^ ((b >> 63) & 0x7fffffffffffffffll);
}
__device__ __forceinline__ double score_of(long long k) {
  return __longlong_as_double(k ^ ((k >> 63) & 0x7fffffffffffffffll));
}
struct __align__(16) Candidate {
  long long key;
  int flat, k;  // k * V + v, and k
};
constexpr long long kNoKey = -0x7fffffffffffffffll - 1;  // (behind every score's)
__device__ __forceinline__ bool better(const Candidate& a, const Candidate& b) {
  return a.key > b.key || (a.key == b.key && a.flat < b.flat);
}
// How many of list[0 .. n) are better than c; four neighbouring lanes share a
// candidate.
__device__ __noinline__ int rank_of(const Candidate c, const Candidate* list, int n) {
  int above = 0;
#pragma unroll 2
  for (int j = threadIdx.x & 3; j < n; j += 4) above += better(list[j], c);
  above += __shfl_xor_sync(kAll, above, 1);
  return above + __shfl_xor_sync(kAll, above, 2);
}

// A living row in vectors: `head` elements in front of the first whole vector,
// `vecs` whole ones, `tail` elements behind them.
template <typename T>
struct Row {
  const T* p;
  int k, head, vecs, tail;
  __device__ __forceinline__ Row(const SelectParams& a, int b, int k) : k(k) {
    p = reinterpret_cast<const T*>(a.logits) + b * a.stride_b + k * a.stride_k;
    const int off = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    constexpr int per = Logits<T>::kPer;
    head = min((per - off) & (per - 1), a.V);
    vecs = (a.V - head) / per;
    tail = a.V - head - vecs * per;
  }
  __device__ __forceinline__ const uint4* vec() const {
    return reinterpret_cast<const uint4*>(p + head);
  }
  // element number of the lane's extra element (lanes 0 .. head + tail - 1 of
  // the row's first unit have one), or -1
  __device__ __forceinline__ int extra(int lane) const {
    return lane < head ? lane : lane < head + tail ? vecs * Logits<T>::kPer + lane : -1;
  }
};

struct SelectShared {
  uint8_t row[kMaxBeams * 32];                // Row of each living beam
  float max[kMaxUnits * 32];                  // block maxima
  float unit_h[kMaxUnits], unit_s[kMaxUnits];
  int unit_at[kMaxUnits];                     // a unit's first vector
  uint8_t unit_r[kMaxUnits];                  // and its row
  float4 rows[kMaxCluster][kMaxBeams];        // every CTA's sums of every row
  double lse[kMaxBeams];                      // inf: no candidates
  float lse32[kMaxBeams], cum[kMaxBeams];
  uint32_t code[kMaxBeams];                   // of the CTA's part of a row, then of the row
  int parts[kParts / 32][kMaxBeams][32];      // maxima of the even and the odd units of every row
  Candidate cand[kMaxCandidates];
  Candidate lists[kMaxCluster * kMaxOut];     // of every CTA, in order (CTA 0's are used)
  int list_count[kMaxCluster];
  Candidate warp_best[kWarps];
  uint16_t list[kMaxUnits * 32];              // blocks that pass the bound
  int blocks, count;
};
static_assert(kCtasPerSm * (sizeof(SelectShared) + 1024) <= 228 << 10, "resident together");

// An fp32 value's order as a whole number.
__device__ __forceinline__ int order32(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}

__device__ __forceinline__ float value32(int i) {
  return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) select_kernel(const SelectParams p) {
  using L = Logits<T>;
  constexpr int per = L::kPer;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  SelectShared& sm = *reinterpret_cast<SelectShared*>(smem_raw);
  Row<T>* const rows = reinterpret_cast<Row<T>*>(sm.row);
  static_assert(sizeof(Row<T>) <= 32, "a row's place");

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int b = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  griddep_launch_dependents();
  griddep_wait();
  // the beams that live: a finite score, and not finished
  float cum = neg_inf();
  bool done = false;
  if (lane < p.K) {
    cum = p.scores[(int64_t)b * p.K + lane];
    done = p.finished != nullptr && p.finished[(int64_t)b * p.K + lane] != 0;
  }
  const bool scored = isfinite(cum);
  const uint32_t live_mask = __ballot_sync(kAll, scored && !done);
  const uint32_t done_mask = __ballot_sync(kAll, scored && done);
  const int live = __popc(live_mask);
  if (warp == 0) {
    if (scored && !done) rows[__popc(live_mask & ((1u << lane) - 1))] = Row<T>(p, b, lane);
    if (lane == 0) sm.blocks = sm.count = 0;
    sm.code[lane] = 0;
  }
  for (int r = warp; r < p.K; r += kWarps)
    sm.parts[0][r][lane] = sm.parts[1][r][lane] = order32(neg_inf());
  __syncthreads();
  cluster_arrive();  // (the others' shared memory is written once they have started)

  // units [u0, u1) of every row are this CTA's: its unit i * live + r is number
  // u0 + i of living row r; a warp takes every kWarps-th, a step at a time
  const int u0 = (int)((int64_t)p.row_units * rank / ranks);
  const int u1 = (int)((int64_t)p.row_units * (rank + 1) / ranks);
  const int units = (u1 - u0) * live;
  struct Place {  // of a step: unit, row, unit in the row, first vector of the step, step in the unit
    int u, r, i, at, s;
  };
  const int row_step = p.steps * kStepVecs;
  auto settle = [&](Place& x) {  // a row behind the last one: the next unit of an earlier one
    while (x.r >= live) {
      x.r -= live;
      x.at += row_step;
      ++x.i;
    }
  };
  auto advance = [&](Place& x) {
    x.at += kStepVecs;
    if (++x.s < p.steps) return;
    x.s = 0;
    x.at -= row_step;
    x.u += kWarps;
    x.r += kWarps;
    settle(x);
  };
  Place now = {warp, warp, 0, u0 * row_step, 0};
  if (units > 0) settle(now);
  Place next = now;
  // the next step's vectors are on their way while a step is computed
  auto load = [&](uint4 (&v)[kVecs]) {
    if (next.u >= units) return;
    const Row<T>& row = rows[next.r];
    const uint4* from = row.vec() + next.at + lane;
    const int left = row.vecs - next.at - lane;
    if (left + lane >= kStepVecs) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) v[j] = load16(from + j * 32);
    } else {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        v[j] = L::none();
        if (j * 32 < left) v[j] = load16(from + j * 32);
      }
    }
    advance(next);
  };
  // (a lane may have thousands of steps: what its sum lacks is carried along)
  float top = neg_inf(), h = kNothing, sum = 0.f, lack = 0.f;
  // (rows that lie a multiple of 16 bytes apart are cut alike; with codes even so 64 x 8
  // beams of 128000 logits took 38.0 us instead of 36.6)
  const bool coded = p.K > 1 && p.stride_k * sizeof(T) % 16 != 0;
  uint32_t code = 0;
  auto compute = [&](const uint4 (&v)[kVecs]) {
    float x_extra = neg_inf();
    if (now.at == 0) {
      const int e = rows[now.r].extra(lane);
      if (e >= 0) {
        x_extra = L::one(rows[now.r].p + e);
        code += L::bits(rows[now.r].p + e) & (std::is_same<T, float>::value ? ~0u : 0x7fffu);
      }
    }
    top = fmaxf(top, fmaxf(L::largest(v), x_extra));
    const Reference ref = reference_of<T>(top);
    const float down = pow4(h - ref.h);
    sum *= down;
    lack *= down;
    h = ref.h;
    const float2 hi = make_float2(ref.hi, ref.hi), lo = make_float2(ref.lo, ref.lo);
    const float2 minus = make_float2(-ref.minus, -ref.minus);
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      float f[per];
      L::expand(v[j], f);
#pragma unroll
      for (int c = 0; c < per; c += 2) {
        const float2 x = make_float2(f[c], f[c + 1]);
        const float2 t = fma2(x, lo, fma2(x, hi, minus));
        acc[c / 2 & 1] = add2(acc[c / 2 & 1], make_float2(ex2(t.x), ex2(t.y)));
      }
    }
    if (coded) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) code = L::code(v[j], code);
    }
    const float2 both = add2(acc[0], acc[1]);
    float step = both.x + both.y;
    if (now.at == 0) step += ex2(fmaf(x_extra, ref.lo, fmaf(x_extra, ref.hi, -ref.minus)));
    const float upto = sum + step, added = upto - sum;
    lack += (sum - (upto - added)) + (step - added);
    sum = upto;
    const int u = now.u, r = now.r, odd = now.i & 1, at = now.at - now.s * kStepVecs;
    advance(now);
    if (now.u == u) return;
    // the unit's maxima, and its sum under the largest of the lanes' references
    sm.max[u * 32 + lane] = top;
    atomicMax(&sm.parts[odd][r][lane], order32(top));
    const float uh = warp_max(h);
    sum = (sum + lack) * pow4(h - uh);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    code = __reduce_add_sync(kAll, code);
    if (lane == 0) {
      atomicAdd(&sm.code[r], code);
      sm.unit_h[u] = uh;
      sm.unit_s[u] = sum;
      sm.unit_at[u] = at;
      sm.unit_r[u] = (uint8_t)r;
    }
    top = neg_inf();
    h = kNothing;
    sum = lack = 0.f;
    code = 0;
  };
  {
    uint4 v[kVecs], w[kVecs];
    load(v);
#pragma unroll 1
    while (now.u < units) {
      load(w);
      compute(v);
      if (now.u >= units) break;
      load(v);
      compute(w);
    }
  }
  __syncthreads();

  // rows: this CTA's sums, given to every CTA of the cluster
  cluster_wait();
#pragma unroll 1
  for (int r = warp; r < live; r += kWarps) {
    Sum s = {kNothing, 0.f, 0.f};
    // (at most two units a lane)
#pragma unroll 1
    for (int u = lane * live + r; u < units; u += 32 * live) {
      const float h = sm.unit_h[u], m = fmaxf(h, s.h);
      const float x = s.hi * pow4(s.h - m), y = sm.unit_s[u] * pow4(h - m);
      const float t = x + y;
      s = {m, t, (x - (t - (t - x))) + (y - (t - x))};
    }
    s = warp_total(s);
    if (lane < ranks)
      *cluster.map_shared_rank(&sm.rows[rank][r], lane) = make_float4(s.h, s.hi, s.lo, __uint_as_float(sm.code[r]));
  }
  cluster.sync();
#pragma unroll 1
  for (int r = warp; r < live; r += kWarps) {
    Sum s = {kNothing, 0.f, 0.f};
    uint32_t part = 0;
    if (lane < ranks) {
      const float4 f = sm.rows[lane][r];
      s = {f.x, f.y, f.z};
      part = __float_as_uint(f.w);
    }
    s = warp_total(s);
    part = __reduce_add_sync(kAll, part);
    const float row_cum = __shfl_sync(kAll, cum, rows[r].k);
    if (lane == 0) {
      // a row without a distribution (NaN or +inf in it, or nothing but -inf) has no candidates
      double lse = INFINITY;
      if (s.hi > 0.f && isfinite(s.hi) && isfinite(s.h)) lse = ln_of(s);
      else if (rank == 0 && s.hi != 0.f) report(p.err, PA_DEVERR_VALUE, b * p.K + rows[r].k, 0);
      sm.lse[r] = lse;
      sm.lse32[r] = (float)lse;
      sm.cum[r] = row_cum;
      // (without the -inf that stand for vectors the row does not have)
      const uint32_t slots = (uint32_t)p.row_units * p.steps * kStepVecs;
      sm.code[r] = part - (slots - rows[r].vecs) * L::code(L::none(), 0);
    }
  }
  __syncthreads();
  if (coded && live > 1) {  // equal rows: the first one's lse
    if (warp == 0) {
      const double lse = lane < live ? sm.lse[lane] : INFINITY;
      const uint32_t same = __match_any_sync(kAll, lane < live ? sm.code[lane] & L::kCode : ~0u);
      const double first = __shfl_sync(kAll, lse, __ffs((int)same) - 1);
      // (each is off by less than 2^-18)
      if (isfinite(first) && fabs(lse - first) <= 0x1p-17 + fabs(first) * 0x1p-50) {
        sm.lse[lane] = first;
        sm.lse32[lane] = (float)first;
      }
    }
    __syncthreads();
  }

  // The bound: the N-th largest of the maxima of kParts parts of the blocks.  A
  // part has blocks of every row (the best beam may be far ahead of the others).
  float bound = neg_inf();
  {
    float size = 0.f, part[2] = {neg_inf(), neg_inf()};
#pragma unroll 1
    for (int r = 0; r < live; ++r) {
      const float lse = sm.lse32[r], s = sm.cum[r];
      if (lse == -neg_inf()) continue;
      size = fmaxf(size, fmaxf(fabsf(lse), fabsf(s)));
      part[0] = fmaxf(part[0], s + (value32(sm.parts[0][r][lane]) - lse));
      part[1] = fmaxf(part[1], s + (value32(sm.parts[1][r][lane]) - lse));
    }
    int even = order32(part[0]), odd = order32(part[1]), top = order32(neg_inf());
    // the largest ones, one value after the other, until N parts have gone
#pragma unroll 1
    for (int gone = 0; gone < p.N;) {
      top = __reduce_max_sync(kAll, max(even, odd));
      if (top <= order32(neg_inf())) break;
      gone += __popc(__ballot_sync(kAll, even == top)) + __popc(__ballot_sync(kAll, odd == top));
      if (even == top) even = order32(neg_inf());
      if (odd == top) odd = order32(neg_inf());
    }
    bound = value32(top);
    // fp32 scores are off by 2^-24 of lse, of x - lse (which is no larger than the
    // score and s together) and of the score; the N-th best element and the blocks
    // that bound it each once
    bound -= fmaxf(size, fabsf(bound)) * 0x1p-20f;
  }
  // (a score of -inf: nothing to choose, or a row without a distribution)
  auto passes = [&](float s) { return s > neg_inf() && s >= bound; };
#pragma unroll 1
  for (int u = warp; u < units; u += kWarps)
    if (const int r = sm.unit_r[u]; passes(sm.cum[r] + (sm.max[u * 32 + lane] - sm.lse32[r])))
      sm.list[atomicAdd(&sm.blocks, 1)] = (uint16_t)(u * 32 + lane);
  __syncthreads();

  // elements of these blocks: 16 lanes a block, or 32 where it has more vectors, one
  // vector each at a time (the loads are misses, one after the other: 8 lanes took
  // 8200 cycles for 33 vectors)
  const int per_block = p.steps * kVecs + 1, lanes_log2 = per_block > 16 ? 5 : 4;
  auto each_element = [&](auto&& f) {  // f(row, element, logit)
#pragma unroll 1
    for (int i = tid >> lanes_log2; i < sm.blocks; i += kThreads >> lanes_log2) {
      const int blk = sm.list[i], u = blk >> 5, l = blk & 31, r = sm.unit_r[u], at = sm.unit_at[u];
      const Row<T>& row = rows[r];
      const float lse = sm.lse32[r], s = sm.cum[r];
#pragma unroll 1
      for (int j = tid & ((1 << lanes_log2) - 1); j < per_block - (at != 0);
           j += 1 << lanes_log2) {
        uint4 v = L::none();
        int e = row.head + (at + j * 32 + l) * per;
        if (j == per_block - 1) {  // the extra element, of a row's first unit
          e = row.extra(l);
          if (e >= 0) v.x = L::alone(row.p + e);
        } else if (at + j * 32 + l < row.vecs) {
          v = load16(row.vec() + at + j * 32 + l);
        }
        float x[per];
        L::expand(v, x);
        uint32_t in = 0;
#pragma unroll
        for (int c = 0; c < per; ++c) in |= passes(s + (x[c] - lse)) ? 1u << c : 0u;
        for (; in != 0; in &= in - 1) {
          const int c = __ffs((int)in) - 1;
          f(r, e + c, L::one(row.p + e + c));
        }
      }
    }
  };
  auto candidate = [&](int r, int e, float x) {
    return Candidate{order_of((double)sm.cum[r] + ((double)x - sm.lse[r])), rows[r].k * p.V + e, rows[r].k};
  };
  each_element([&](int r, int e, float x) {
    const int at = atomicAdd(&sm.count, 1);
    if (at < kMaxCandidates) sm.cand[at] = candidate(r, e, x);
  });
  __syncthreads();

  // the CTA's best, in order, to CTA 0
  Candidate* const lists = cluster.map_shared_rank(sm.lists, 0) + rank * p.N;
  const int count = sm.count;
  if (count <= kMaxCandidates) {
#pragma unroll 1
    for (int i0 = 0; i0 < count; i0 += kThreads / 4) {
      const int i = i0 + tid / 4;
      const Candidate c = sm.cand[min(i, count - 1)];
      const int above = rank_of(c, sm.cand, count);
      if (i < count && above < p.N && (tid & 3) == 0) lists[above] = c;
    }
  } else {
    // too many: the best one behind the last one found, N times
    Candidate last = {0x7fffffffffffffffll, -1, 0};
    for (int out = 0; out < p.N; ++out) {
      Candidate best = {kNoKey, 0x7fffffff, 0};
      each_element([&](int r, int e, float x) {
        const Candidate c = candidate(r, e, x);
        if (better(last, c) && better(c, best)) best = c;
      });
      auto fold = [&](int o) {
        const Candidate c = {__shfl_xor_sync(kAll, best.key, o), __shfl_xor_sync(kAll, best.flat, o),
                             __shfl_xor_sync(kAll, best.k, o)};
        if (better(c, best)) best = c;
      };
      for (int o = 16; o > 0; o >>= 1) fold(o);
      if (lane == 0) sm.warp_best[warp] = best;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w)
        if (better(sm.warp_best[w], best)) best = sm.warp_best[w];
      if (tid == 0) lists[out] = best;
      last = best;  // (more than kMaxCandidates pass, so there is one)
      __syncthreads();
    }
  }
  if (tid == 0) *cluster.map_shared_rank(&sm.list_count[rank], 0) = min(count, p.N);
  cluster_arrive();
  if (rank != 0) return;
  cluster_wait();

  // One warp joins the lists: lane c has the first candidate left of CTA c's, and
  // that of beam c if it is finished; the best of all, N times.
  if (warp != 0) return;
  const int64_t out0 = (int64_t)b * p.N;
  const Candidate none = {kNoKey, 0x7fffffff, 0};
  const Candidate* head = sm.lists + lane * p.N;
  int left = lane < ranks ? sm.list_count[lane] : 0;
  Candidate a = left > 0 ? *head : none;
  Candidate f = none;
  if (done_mask >> lane & 1) f = {order_of((double)cum), lane * p.V + p.end_token, lane};
#pragma unroll 1
  for (int out = 0; out < p.N; ++out) {
    const bool end = better(f, a);
    const Candidate c = end ? f : a;
    // the largest key, its high word first, then the lowest place
    const int hi = (int)(c.key >> 32), top = __reduce_max_sync(kAll, hi);
    const uint32_t lo = hi == top ? (uint32_t)c.key : 0u, low = __reduce_max_sync(kAll, lo);
    const int at = hi == top && lo == low ? c.flat : 0x7fffffff;
    if (at == __reduce_min_sync(kAll, at) && hi == top && lo == low && c.key != kNoKey) {
      const int v = c.flat - c.k * p.V;
      p.scores_out[out0 + out] = (float)score_of(c.key);
      p.parents[out0 + out] = c.k;
      p.tokens[out0 + out] = v;
      if (p.finished_out != nullptr)
        p.finished_out[out0 + out] = v == p.end_token || (done_mask >> c.k & 1);
      if (end) {
        f = none;
      } else {
        ++head;
        a = --left > 0 ? *head : none;
      }
    } else if (top == (int)(kNoKey >> 32) && low == 0 && lane == 0) {  // nothing is left
      p.scores_out[out0 + out] = neg_inf();
      p.parents[out0 + out] = p.tokens[out0 + out] = -1;
      if (p.finished_out != nullptr) p.finished_out[out0 + out] = 0;
    }
  }
}

template <typename T>
cudaError_t launch_select(SelectParams p, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  static std::atomic<int> resident[64][kClusterLimit + 1];  // by device and size; 0: not known
  constexpr int per = 16 / (int)sizeof(T);
  const int vecs = p.V / per + 1;
  const int steps = (vecs + kStepVecs - 1) / kStepVecs;  // of a row
  // CTAs of a request: as many as let all requests be resident together, with a
  // step of a row for each.  (Where they are not, one each.)
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(SelectShared);
  cfg.stream = st;
  cudaLaunchAttribute attrs[2] = {};
  cudaLaunchAttribute& at = attrs[0];
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  overlap_launch(&attrs[1]);
  cfg.attrs = attrs;
  cfg.numAttrs = 1;
  const cudaError_t e = allow_shared(reinterpret_cast<const void*>(select_kernel<T>),
                                     (int)sizeof(SelectShared), &allowed);
  if (e != cudaSuccess) return e;
  int ctas = steps < kMaxCluster ? steps : kMaxCluster;
  while (ctas > 1) {
    cfg.gridDim = dim3((unsigned)ctas);
    at.val.clusterDim.x = (unsigned)ctas;
    if (p.B <= resident_clusters(select_kernel<T>, cfg, ctas, resident)) break;
    --ctas;
  }
  // a unit has as few steps as let the CTA's maxima fit
  p.steps = 1;
  for (;;) {
    p.row_units = (vecs + p.steps * kStepVecs - 1) / (p.steps * kStepVecs);
    if ((int64_t)((p.row_units + ctas - 1) / ctas) * p.K <= kMaxUnits) break;
    ++p.steps;
  }
  cfg.gridDim = dim3((unsigned)(p.B * ctas));
  at.val.clusterDim.x = (unsigned)ctas;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_kernel<T>, p);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" PA_API int pa_beam_select(const void* logits, int64_t stride_b, int64_t stride_k,
                                     const float* scores, const uint8_t* finished, int end_token,
                                     int B, int K, int V, int N, float* scores_out,
                                     int32_t* parents, int32_t* tokens, uint8_t* finished_out,
                                     int32_t* err_word, int dtype, pa_stream_t stream) {
  if (dtype != PA_F16 && dtype != PA_BF16 && dtype != PA_F32)
    return set_error(PA_ERR_UNSUPPORTED, "dtype %d", dtype);
  if (B < 0 || K < 1 || V < 1 || N < 1)
    return set_error(PA_ERR_INVALID_ARG, "B must be >= 0; K, V and N >= 1");
  if (K > kMaxBeams) return set_error(PA_ERR_UNSUPPORTED, "more than %d beams", kMaxBeams);
  if (N > kMaxOut) return set_error(PA_ERR_UNSUPPORTED, "more than %d candidates", kMaxOut);
  if (V > (1 << 24)) return set_error(PA_ERR_UNSUPPORTED, "a vocabulary of more than 2^24");
  if (B > (1 << 20)) return set_error(PA_ERR_UNSUPPORTED, "more than 2^20 requests");
  if (B == 0) return PA_OK;
  if (logits == nullptr || scores == nullptr || scores_out == nullptr || parents == nullptr ||
      tokens == nullptr)
    return set_error(PA_ERR_INVALID_ARG,
                     "logits, scores, scores_out, parents and tokens must be non-NULL");
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == PA_F32 ? 4 : 2) != 0)
    return set_error(PA_ERR_INVALID_ARG, "logits must be aligned to its elements");
  if (stride_b < 0 || stride_k < 0)
    return set_error(PA_ERR_INVALID_ARG, "negative strides");
  if (end_token >= V || (finished != nullptr && end_token < 0))
    return set_error(PA_ERR_INVALID_ARG, "end_token must be a token of the vocabulary");
  if (scores_out == scores || (finished != nullptr && finished_out == finished))
    return set_error(PA_ERR_INVALID_ARG, "scores and finished may not be replaced");
  SelectParams p{};
  p.logits = logits;
  p.stride_b = stride_b;
  p.stride_k = stride_k;
  p.scores = scores;
  p.finished = finished;
  p.end_token = end_token < 0 ? -1 : end_token;
  p.B = B;
  p.K = K;
  p.V = V;
  p.N = N;
  p.scores_out = scores_out;
  p.parents = parents;
  p.tokens = tokens;
  p.finished_out = finished_out;
  p.err = err_word;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == PA_F16    ? launch_select<__half>(p, st)
                        : dtype == PA_BF16 ? launch_select<__nv_bfloat16>(p, st)
                                           : launch_select<float>(p, st);
  if (e != cudaSuccess) return set_error(PA_ERR_CUDA, "select launch: %s", cudaGetErrorString(e));
  return PA_OK;
}
