// A beam search's selection over beams and vocabulary (sm_103a): from the logits
// of every beam the best continuations of each request (pa_beam_select).
//
// Mathematics.  Beam k of a request has the score s_k and the logits x_k[v]:
//   lse_k = ln sum_v exp(x_k[v]),   score(k, v) = s_k + (x_k[v] - lse_k),
// and the N largest scores over all (k, v) are wanted, in order, the lowest
// k * V + v first among equal ones.  exp is taken as 2^(x log2(e) - n) against
// a whole number n, so that sums under different references are brought
// together by exact powers of two; log2(e) is a sum of two fp32 values, which
// leaves one rounding of the exponent.  lse and the scores of the candidates
// are in 64 bits: next to the border candidates of different beams lie so close
// that 32 bits would often choose another one.
//
// One pass over the logits.  A lane reads its elements once, in registers: their
// maximum, then their sum.  Only the maxima are kept (one in 64 or more
// elements, in shared memory).  The N largest elements lie in blocks whose
// maximum is among the N largest maxima, so a bound found from the maxima
// leaves a few dozen blocks, whose elements are read once more (from L2) and
// ranked.  Where more elements than fit pass the bound (many equal logits), the
// N best are found one after the other.
//
// A cluster of up to 16 CTAs per request: the beams of a request must be
// compared with one another, and over distributed shared memory that takes two
// barriers, no scratch memory and no second launch.  Every row is dealt over the
// CTAs in the same way, so equal rows have bitwise equal sums and their ties go
// to the lower index.
#include <cooperative_groups.h>

#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace cg = cooperative_groups;

namespace pa {
int set_error(int code, const char* fmt, ...);

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 8;           // 16-byte vectors of a lane in a step
constexpr int kMaxBeams = 32;
constexpr int kMaxOut = 64;
constexpr int kParts = 64;         // of the block maxima: the N-th largest of their maxima is the bound
constexpr int kMaxCandidates = 1024;
constexpr int kMaxCluster = 16;
constexpr int kMaxUnits = 320;     // of a CTA: 40 KB of block maxima

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
  int steps;      // steps of kVecs vectors in a unit
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
  static __device__ __forceinline__ float one(const T* p) {
    if constexpr (std::is_same<T, float>::value) return __ldg(p);
    else return (float)*p;
  }
};

// Larger is better; a score's order as a whole number (+0 and -0 alike).
__device__ __forceinline__ long long order_of(double s) {
  const long long b = __double_as_longlong(s + 0.0);
  return b ^ ((b >> 63) & 0x7fffffffffffffffll);
}
__device__ __forceinline__ double score_of(long long k) {
  return __longlong_as_double(k ^ ((k >> 63) & 0x7fffffffffffffffll));
}
struct Candidate {
  long long key;
  int flat;  // k * V + v; < 0: none
  int pad;
};
__device__ __forceinline__ bool better(long long ka, int fa, long long kb, int fb) {
  return ka > kb || (ka == kb && fa < fb);
}

// 2^d for a whole d <= 0 (0 below the normal range).
__device__ __forceinline__ float pow2_whole(float d) {
  return d < -126.f ? 0.f : __int_as_float((127 + (int)d) << 23);
}

// The shape of row k in vectors: `head` elements in front of the first whole
// vector, `vecs` whole ones, `tail` elements behind them.
template <typename T>
struct Row {
  const T* p;
  int head, vecs, tail;
  __device__ __forceinline__ Row(const SelectParams& a, int b, int k) {
    p = reinterpret_cast<const T*>(a.logits) + b * a.stride_b + k * a.stride_k;
    const int off = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    constexpr int per = Logits<T>::kPer;
    head = min((per - off) % per, a.V);
    vecs = (a.V - head) / per;
    tail = a.V - head - vecs * per;
  }
  // element number of the lane's extra element (lanes 0 .. head + tail - 1 of
  // the row's first unit have one), or -1
  __device__ __forceinline__ int extra(int lane) const {
    return lane < head ? lane : lane < head + tail ? head + vecs * Logits<T>::kPer + lane - head : -1;
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) select_kernel(const SelectParams p) {
  using L = Logits<T>;
  constexpr int per = L::kPer;
  extern __shared__ float s_max[];  // [units of the CTA][32] block maxima
  __shared__ float s_unit_n[kMaxUnits], s_unit_s[kMaxUnits];
  __shared__ float s_row_n[kMaxCluster][kMaxBeams];   // every CTA's sums of every row
  __shared__ double s_row_s[kMaxCluster][kMaxBeams];
  __shared__ double s_base[kMaxBeams];
  __shared__ float s_base32[kMaxBeams];
  __shared__ int s_live[kMaxBeams];
  __shared__ float s_part[kParts];
  __shared__ float s_bound;
  __shared__ int s_blocks, s_count;
  __shared__ uint16_t s_list[kMaxUnits * 32];  // blocks that pass the bound
  __shared__ Candidate s_cand[kMaxCandidates + kMaxBeams];
  __shared__ Candidate s_best[kMaxOut];
  __shared__ Candidate s_warp[kWarps];

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int b = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // the beams that live: a finite score, and not finished
  float cum = neg_inf();
  bool done = false;
  if (lane < p.K) {
    cum = p.scores[(int64_t)b * p.K + lane];
    done = p.finished != nullptr && p.finished[(int64_t)b * p.K + lane] != 0;
  }
  const bool scored = isfinite(cum);
  const uint32_t live_mask = __ballot_sync(0xffffffffu, scored && !done);
  const uint32_t done_mask = __ballot_sync(0xffffffffu, scored && done);
  const int live = __popc(live_mask);
  if (warp == 0 && scored && !done) s_live[__popc(live_mask & ((1u << lane) - 1))] = lane;
  if (tid == 0) s_blocks = s_count = 0;
  __syncthreads();
  cluster_arrive();  // (the others' shared memory is written once they have started)

  // units [u0, u1) of every row are this CTA's: unit i * live + r is number
  // u0 + i of living row r
  const int u0 = (int)((int64_t)p.row_units * rank / ranks);
  const int u1 = (int)((int64_t)p.row_units * (rank + 1) / ranks);
  const int units = (u1 - u0) * live;
  const int unit_vecs = p.steps * kVecs * 32;

  for (int u = warp; u < units; u += kWarps) {
    const int i = u / live, r = u - i * live;
    const Row<T> row(p, b, s_live[r]);
    const uint4* vec = reinterpret_cast<const uint4*>(row.p + row.head);
    float top = neg_inf(), n = 0.f, sum = 0.f;
    for (int s = 0; s < p.steps; ++s) {
      const int at = (u0 + i) * unit_vecs + s * kVecs * 32 + lane;
      uint4 v[kVecs];
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        v[j] = L::none();
        if (at + j * 32 < row.vecs) v[j] = load16(vec + at + j * 32);
      }
      float x_extra = neg_inf();
      if (s == 0 && u0 + i == 0) {
        const int e = row.extra(lane);
        if (e >= 0) x_extra = L::one(row.p + e);
      }
      float m = x_extra;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        float f[per];
        L::expand(v[j], f);
#pragma unroll
        for (int c = 0; c < per; ++c) m = fmaxf(m, f[c]);
      }
      const float was = top;
      top = fmaxf(top, m);
      const float ref = top == neg_inf() ? 0.f : rintf(top * kLog2eHi);
      if (was != neg_inf()) sum *= pow2_whole(n - ref);
      n = ref;
      auto add = [&](float x) { sum += ex2(fmaf(x, kLog2eLo, fmaf(x, kLog2eHi, -n))); };
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        float f[per];
        L::expand(v[j], f);
#pragma unroll
        for (int c = 0; c < per; ++c) add(f[c]);
      }
      add(x_extra);
    }
    s_max[u * 32 + lane] = top;
    // the unit's sum, under the largest of the lanes' references (a lane that
    // holds nothing but -inf has a sum of zero or NaN)
    float un = top == neg_inf() ? neg_inf() : n;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) un = fmaxf(un, __shfl_xor_sync(0xffffffffu, un, o));
    if (un != neg_inf() && top != neg_inf()) sum *= pow2_whole(n - un);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      s_unit_n[u] = un;
      s_unit_s[u] = sum;
    }
  }
  __syncthreads();

  // rows: this CTA's sums, given to every CTA of the cluster
  cluster_wait();
  for (int r = warp; r < live; r += kWarps) {
    float rn = neg_inf();
    for (int i = lane; i < u1 - u0; i += 32) rn = fmaxf(rn, s_unit_n[i * live + r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) rn = fmaxf(rn, __shfl_xor_sync(0xffffffffu, rn, o));
    double rs = 0;
    for (int i = lane; i < u1 - u0; i += 32) {
      const float un = s_unit_n[i * live + r];
      const float f = un == neg_inf() ? 1.f : pow2_whole(un - rn);
      rs += (double)(s_unit_s[i * live + r] * f);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) rs += __shfl_xor_sync(0xffffffffu, rs, o);
    if (lane < ranks) {
      *cluster.map_shared_rank(&s_row_n[rank][r], lane) = rn;
      *cluster.map_shared_rank(&s_row_s[rank][r], lane) = rs;
    }
  }
  cluster.sync();
  if (warp == 0 && lane < live) {
    float rn = neg_inf();
    for (int c = 0; c < ranks; ++c) rn = fmaxf(rn, s_row_n[c][lane]);
    double rs = 0;
    for (int c = 0; c < ranks; ++c) {
      const float cn = s_row_n[c][lane];
      rs += s_row_s[c][lane] * (double)(cn == neg_inf() ? 1.f : pow2_whole(cn - rn));
    }
    const int k = s_live[lane];
    // a row without a distribution (NaN or +inf in it, or nothing but -inf) has no candidates
    double base = -INFINITY;
    if (rs > 0 && isfinite(rs) && isfinite(rn))
      base = (double)p.scores[(int64_t)b * p.K + k] - ((double)rn * kLn2d + log(rs));
    else if (rank == 0 && (rn != neg_inf() || rs != 0))
      report(p.err, PA_DEVERR_VALUE, b * p.K + k, 0);
    s_base[lane] = base;
    s_base32[lane] = (float)base;
  }
  __syncthreads();

  // the bound: N-th largest of the maxima of kParts parts of the blocks
  const int blocks = units * 32;
  auto block_score = [&](int blk) {
    const int u = blk >> 5;
    return s_base32[u - u / live * live] + s_max[blk];
  };
  {
    float m = neg_inf();
    for (int i = tid; i < blocks; i += kThreads) {
      const float s = block_score(i);
      m = fmaxf(m, s);
    }
    constexpr int each = kThreads / kParts;
#pragma unroll
    for (int o = each / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (tid % each == 0) s_part[tid / each] = m;
  }
  __syncthreads();
  if (tid < kParts) {
    const float m = s_part[tid];
    int above = 0;
    for (int i = 0; i < kParts; ++i) above += s_part[i] > m || (s_part[i] == m && i < tid);
    if (above == p.N - 1) {
      // fp32 scores are off by 2^-24 of the base and of the sum; the N-th best
      // element and the blocks that bound it each once
      float size = fabsf(m);
      for (int r = 0; r < live; ++r)
        if (s_base32[r] > neg_inf()) size = fmaxf(size, fabsf(s_base32[r]));
      s_bound = m - size * 0x1p-21f;
    }
  }
  __syncthreads();
  const float bound = s_bound;
  // (a score of -inf: nothing to choose, or a row without a distribution)
  auto passes = [&](float s) { return s > neg_inf() && s >= bound; };
  for (int i = tid; i < blocks; i += kThreads)
    if (passes(block_score(i))) s_list[atomicAdd(&s_blocks, 1)] = (uint16_t)i;
  __syncthreads();

  // elements of these blocks, one vector a thread
  const int per_block = p.steps * kVecs + 1;
  auto take = [&](int r, float x, int e) {
    if (!passes(s_base32[r] + x)) return;
    const int at = atomicAdd(&s_count, 1);
    if (at < kMaxCandidates)
      s_cand[at] = {order_of(s_base[r] + (double)x), s_live[r] * p.V + e, 0};
  };
  // every element of vector j (the last one: the extra element) of a block
  auto each_of = [&](int blk, int j, auto&& f) {
    const int u = blk >> 5, l = blk & 31, i = u / live, r = u - i * live;
    const Row<T> row(p, b, s_live[r]);
    if (j == per_block - 1) {
      const int e = u0 + i == 0 ? row.extra(l) : -1;
      if (e >= 0) f(r, L::one(row.p + e), e);
      return;
    }
    const int at = (u0 + i) * unit_vecs + j * 32 + l;
    if (at >= row.vecs) return;
    const uint4 v = load16(reinterpret_cast<const uint4*>(row.p + row.head) + at);
    float x[per];
    L::expand(v, x);
#pragma unroll
    for (int c = 0; c < per; ++c) f(r, x[c], row.head + at * per + c);
  };
  for (int w = tid; w < s_blocks * per_block; w += kThreads)
    each_of(s_list[w / per_block], w % per_block, take);
  __syncthreads();

  int count = s_count;
  if (count <= kMaxCandidates) {
    if (tid < p.N) s_best[tid] = {0, -1, 0};
    __syncthreads();
    for (int i = tid; i < count; i += kThreads) {
      const Candidate c = s_cand[i];
      int above = 0;
      for (int j = 0; j < count && above < p.N; ++j)
        above += better(s_cand[j].key, s_cand[j].flat, c.key, c.flat);
      if (above < p.N) s_best[above] = c;
    }
  } else {
    // too many: the best one behind the last one found, N times
    Candidate last = {0x7fffffffffffffffll, -1, 0};
    for (int out = 0; out < p.N; ++out) {
      Candidate best = {0, -1, 0};
      auto look = [&](int r, float x, int e) {
        if (!passes(s_base32[r] + x)) return;
        const long long key = order_of(s_base[r] + (double)x);
        const int flat = s_live[r] * p.V + e;
        if (!better(last.key, last.flat, key, flat)) return;
        if (best.flat < 0 || better(key, flat, best.key, best.flat)) best = {key, flat, 0};
      };
      for (int w = tid; w < s_blocks * per_block; w += kThreads)
        each_of(s_list[w / per_block], w % per_block, look);
      auto fold = [&](int o) {
        const long long key = __shfl_xor_sync(0xffffffffu, best.key, o);
        const int flat = __shfl_xor_sync(0xffffffffu, best.flat, o);
        if (flat >= 0 && (best.flat < 0 || better(key, flat, best.key, best.flat)))
          best = {key, flat, 0};
      };
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) fold(o);
      if (lane == 0) s_warp[warp] = best;
      __syncthreads();
      best = lane < kWarps ? s_warp[lane] : Candidate{0, -1, 0};
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) fold(o);
      if (tid == 0) s_best[out] = best;
      last = best;
      __syncthreads();
      if (best.flat < 0) {  // (uniform) nothing is left
        for (int i = out + 1 + tid; i < p.N; i += kThreads) s_best[i] = best;
        break;
      }
    }
  }
  cluster.sync();  // every CTA's best; and the candidates of CTA 0 are no longer read

  if (rank == 0) {
    // the lists of all CTAs, and one candidate of each finished beam
    const int all = ranks * p.N;
    for (int i = tid; i < all; i += kThreads)
      s_cand[i] = cluster.map_shared_rank(s_best, i / p.N)[i % p.N];
    if (tid < kMaxBeams) {
      Candidate c = {0, -1, 0};
      if (tid < p.K && (done_mask >> tid & 1))
        c = {order_of((double)cum), tid * p.V + p.end_token, 0};
      s_cand[all + tid] = c;
    }
  }
  cluster.sync();  // (no CTA leaves while its list is read)
  if (rank != 0) return;
  const int all = ranks * p.N + kMaxBeams;
  const int64_t out0 = (int64_t)b * p.N;
  int here = 0;
  for (int i = tid; i < all; i += kThreads) {
    const Candidate c = s_cand[i];
    if (c.flat < 0) continue;
    ++here;
    int above = 0;
    for (int j = 0; j < all && above < p.N; ++j)
      above += s_cand[j].flat >= 0 && better(s_cand[j].key, s_cand[j].flat, c.key, c.flat);
    if (above >= p.N) continue;
    const int k = c.flat / p.V, v = c.flat - k * p.V;
    p.scores_out[out0 + above] = (float)score_of(c.key);
    p.parents[out0 + above] = k;
    p.tokens[out0 + above] = v;
    if (p.finished_out != nullptr)
      p.finished_out[out0 + above] = v == p.end_token || (done_mask >> k & 1);
  }
  // places without a candidate
  here = __reduce_add_sync(0xffffffffu, here);
  if (tid == 0) s_count = 0;
  __syncthreads();
  if (lane == 0) atomicAdd(&s_count, here);
  __syncthreads();
  for (int i = s_count + tid; i < p.N; i += kThreads) {
    p.scores_out[out0 + i] = neg_inf();
    p.parents[out0 + i] = p.tokens[out0 + i] = -1;
    if (p.finished_out != nullptr) p.finished_out[out0 + i] = 0;
  }
}

template <typename T>
cudaError_t launch_select(SelectParams p, cudaStream_t st) {
  static std::atomic<uint64_t> asked{0}, wide{0}, allowed{0};
  constexpr int per = 16 / (int)sizeof(T);
  const int vecs = p.V / per + 1;
  // CTAs of a request: as many as are resident together (two an SM), with a step
  // of a row for each
  int ctas = 1;
  while (ctas < kMaxCluster && (int64_t)p.B * ctas * 2 <= 2 * num_sms() &&
         (vecs + kVecs * 32 - 1) / (kVecs * 32) >= 2 * ctas)
    ctas *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = allow_shared(reinterpret_cast<const void*>(select_kernel<T>),
                                     kMaxUnits * 32 * (int)sizeof(float), &allowed);
  if (e != cudaSuccess) return e;
  for (;;) {
    // a unit has as few steps as let the CTA's maxima fit
    p.steps = 1;
    for (;;) {
      p.row_units = (vecs + p.steps * kVecs * 32 - 1) / (p.steps * kVecs * 32);
      if ((int64_t)((p.row_units + ctas - 1) / ctas) * p.K <= kMaxUnits) break;
      ++p.steps;
    }
    cfg.dynamicSmemBytes = (size_t)((p.row_units + ctas - 1) / ctas) * p.K * 32 * sizeof(float);
    cfg.gridDim = dim3((unsigned)(p.B * ctas));
    at.val.clusterDim.x = (unsigned)ctas;
    if (ctas <= 8 || wide_clusters(select_kernel<T>, cfg, &asked, &wide)) break;
    ctas = 8;
  }
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
