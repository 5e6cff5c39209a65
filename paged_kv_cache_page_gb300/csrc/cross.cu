// Attention of a ragged batch's rows to the keys of their entry, of another
// length (pa_fwd_cross; sm_103a): the kernel for few rows a kv head, as the beams
// of a request have them, and the entry point.
//
// Mathematics.  O = softmax(scale Q K^T) V over the keys of the entry that are not
// masked, in one pass: a running maximum m and sum l of 2^(s - m), s the scores
// times scale log2(e); O is brought to a new maximum only where P would pass a limit
// of its type otherwise (Range).  Partial results (O, m, l) of different keys are
// joined exactly.
//
// What bounds it is the read of K and V, once for all rows of the entry.  The
// G query heads of a kv head and the rows are packed into tiles of 16 rows, the M
// of mma.sync m16n8k16; P passes from one product to the other in registers.
// Each of a CTA's four warps has its own kv head and its own ring of two
// 8 KB stages, filled by TMA and refilled as soon as the warp has read a stage:
// no wait between warps, and neighbouring heads (which lie behind one another in
// a row of k) are read at about the same time.  Where there are fewer than four
// kv heads the warps of a head take turns over its tiles.  A cluster of up to 16
// CTAs divides the keys where there are few entries; the parts are joined over
// distributed shared memory, so there is no scratch memory and no second launch.
// A ring that the warps share was 1.6 times slower.  Measured: 32 entries of 5 rows
// and 100 to 1500 keys, 16 heads of 64: 23.2 us (4.5 TB/s); 64 of one row and 4096
// keys, 32/8 heads of 128: 159 us (6.7 TB/s); one of 4 rows and 1000 keys, 12 heads of
// 64: 6.4 us, most of it launch, first keys and join.
#include "cross.cuh"

#include <cooperative_groups.h>

#include <atomic>
#include <cmath>
#include <type_traits>

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;
constexpr int kStageBytes = 8192;  // K and V of a tile of one head
constexpr int kRows = 16;          // packed rows of an entry and kv head
constexpr int kCtasPerSm = 3;
constexpr int kMaxCluster = kClusterLimit;

// The largest score is brought to 2^kShift, and may pass that by 2^kSlack before O is
// brought to a new maximum.  fp16 has no numbers below 2^-24, and l counts the P that
// vanish: so the largest is 2^8 at first and 2^15 at most, and keys of 2^-30 of its
// weight still count.
template <typename T> struct Range;
template <> struct Range<__half> {
  static constexpr float kShift = 8.f, kSlack = 7.f;
};
template <> struct Range<__nv_bfloat16> {
  static constexpr float kShift = 0.f, kSlack = 8.f;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A CTA's warps have hs neighbouring kv heads.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    cross_kernel(const __grid_constant__ CrossParams p, const int hs,
                 const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  using E = Elem<T>;
  using R = Range<T>;
  constexpr int TK = cross_narrow_box(D);  // keys of a tile
  constexpr int NT = TK / 8;               // its n-tiles
  constexpr int KD = D / 16;               // k-steps of Q K^T
  constexpr int ND = D / 8;                // n-tiles of P V
  constexpr int kSlab = TK * 128;          // 64 columns of K or V
  constexpr int kTensor = kSlab * (D / 64);
  static_assert(2 * kTensor == kStageBytes, "a stage holds K and V of a tile");
  static_assert(kRows * (D + 2) * 4 <= kStages * kStageBytes, "partial results fit in a ring");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint64_t s_full[kWarps][kStages];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  griddep_launch_dependents();
  griddep_wait();
  // cluster -> entry, group of heads
  const int item = blockIdx.x / ranks;
  const int groups = p.Hkv / hs;
  const int b = item / groups, h = (item - b * groups) * hs + warp % hs;
  const int slice = warp / hs, slices = kWarps / hs;
  const CrossEntry e = cross_entry(p, b, tid == 0 && rank == 0 && item % groups == 0);
  const int rows = e.rows * p.G;
  if (rows <= 0) return;  // (the whole cluster)

  // this warp's tiles: `slices` warps take turns over the CTA's part
  const int tiles = (e.keys + TK - 1) / TK;
  const int t_end = (int)((long long)tiles * (rank + 1) / ranks);
  const int t_begin = (int)((long long)tiles * rank / ranks) + slice;
  const int n = t_begin < t_end ? (t_end - t_begin + slices - 1) / slices : 0;

  uint8_t* ring = smem + warp * kStages * kStageBytes;
  uint64_t* full = s_full[warp];
  const uint64_t policy = l2_policy_evict_first();
  auto fill = [&](int i) {  // by one lane
    const int s = i % kStages, key = e.k0 + (t_begin + i * slices) * TK;
    mbar_arrive_expect_tx(&full[s], kStageBytes);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      tma_load_4d(ring + s * kStageBytes + c * kSlab, &tmk, &full[s], c * 64, h, key, 0, policy);
      tma_load_4d(ring + s * kStageBytes + kTensor + c * kSlab, &tmv, &full[s], c * 64, h, key, 0,
                  policy);
    }
  };
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
    fence_proxy_async_smem();
    for (int i = 0; i < min(n, kStages); ++i) fill(i);
  }
  __syncwarp();

  // Q as the A operand; packed row r is query head h * G + r % G of row r / G
  uint32_t qf[KD][4];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = half * 8 + lane / 4;
    const int at = r / p.G, g = r - at * p.G;
    const T* src = reinterpret_cast<const T*>(p.q) + (int64_t)(e.q0 + at) * p.q_st +
                   (int64_t)(h * p.G + g) * p.q_sh + 2 * (lane & 3);
#pragma unroll
    for (int k = 0; k < KD; ++k)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        qf[k][2 * c + half] =
            r < rows ? __ldg(reinterpret_cast<const uint32_t*>(src + k * 16 + c * 8)) : 0u;
  }

  float o[ND][4], m_use[2], l[2];
#pragma unroll
  for (int i = 0; i < ND; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
  m_use[0] = m_use[1] = neg_inf();
  l[0] = l[1] = 0.f;
  // The lane's key of tile i: its mask is read two tiles ahead and looked at only
  // then (while the memory is busy with K and V a byte takes as long as a tile).
  auto key_of = [&](int i) { return (t_begin + i * slices) * TK + lane; };
  auto mask_of = [&](int i) -> uint32_t {
    if (p.key_mask == nullptr || i >= n || lane >= TK || key_of(i) >= e.keys) return 1;
    return load_byte(p.key_mask + e.k0 + key_of(i));
  };
  constexpr uint32_t kAllKeys = TK == 32 ? 0xffffffffu : (1u << TK) - 1;
  bool ok = true;
  uint32_t mask0 = mask_of(0), mask1 = mask_of(1);

  int i = 0;
  for (; i < n && ok; ++i) {
    const int s = i % kStages;
    const uint32_t bits =
        __ballot_sync(0xffffffffu, lane < TK && key_of(i) < e.keys && mask0 != 0);
    mask0 = mask1;
    mask1 = mask_of(i + 2);
    if (!mbar_wait(&full[s], (uint32_t)(i / kStages & 1))) {
      report(p.err, PA_DEVERR_TIMEOUT, b, 80);
      ok = false;
    }
    ok = __all_sync(0xffffffffu, ok);
    const uint32_t sk = smem_u32(ring + s * kStageBytes), sv = sk + kTensor;

    // S = Q K^T
    float sc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) sc[j][c] = 0.f;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int k = 0; k < KD; k += 2) {
        // matrices: 8 keys by columns 16 k + 8 x, x = lane / 8
        const int key = j * 8 + (lane & 7), col = k * 2 + (lane >> 3);
        uint32_t r[4];
        ldsm4(r, sk + (col >> 3) * kSlab + key * 128 + (((col & 7) ^ (key & 7)) << 4));
        mma<T>(sc[j], qf[k], r[0], r[1]);
        mma<T>(sc[j], qf[k + 1], r[2], r[3]);
      }

    // scores of unseen keys
    if (bits != kAllKeys) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if ((bits >> (j * 8 + 2 * (lane & 3) + c) & 1) == 0) sc[j][c] = sc[j][c + 2] = neg_inf();
    }
    uint32_t pf[NT / 2][4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float top = neg_inf();
#pragma unroll
      for (int j = 0; j < NT; ++j) top = fmaxf(top, fmaxf(sc[j][2 * half], sc[j][2 * half + 1]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      top *= p.scale_log2;
      float& mu = m_use[half];
      const bool lift = top > mu + (R::kShift + R::kSlack) || (mu == neg_inf() && top != neg_inf());
      if (__any_sync(0xffffffffu, lift)) {
        const float to = top - R::kShift, f = lift ? ex2(mu - to) : 1.f;
        if (lift) mu = to;
        l[half] *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          o[d][2 * half] *= f;
          o[d][2 * half + 1] *= f;
        }
      }
      const float ref = mu == neg_inf() ? 0.f : -mu;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float a = ex2(fmaf(sc[j][2 * half], p.scale_log2, ref));
        const float c = ex2(fmaf(sc[j][2 * half + 1], p.scale_log2, ref));
        sum += a + c;
        pf[j / 2][(j & 1) * 2 + half] = E::from_f2(a, c);
      }
      l[half] += sum;
    }

    // O += P V
#pragma unroll
    for (int k = 0; k < NT / 2; ++k)
#pragma unroll
      for (int d = 0; d < ND; d += 2) {
        // matrices: keys 16 k + 8 (x & 1), columns 8 (d + x / 2), x = lane / 8
        const int key = k * 16 + (lane >> 3 & 1) * 8 + (lane & 7), col = d + (lane >> 4);
        uint32_t r[4];
        ldsm4t(r, sv + (col >> 3) * kSlab + key * 128 + (((col & 7) ^ (key & 7)) << 4));
        if (bits != kAllKeys) {
          // (0 times what an unseen key holds, which may be NaN)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t two = bits >> (k * 16 + x * 8 + 2 * (lane & 3));
            const uint32_t keep = ((two & 1) ? 0xffffu : 0u) | ((two & 2) ? 0xffff0000u : 0u);
            r[x] &= keep;
            r[x + 2] &= keep;
          }
        }
        mma<T>(o[d], pf[k], r[0], r[1]);
        mma<T>(o[d + 1], pf[k], r[2], r[3]);
      }
    __syncwarp();  // the stage has been read by every lane
    if (lane == 0 && ok && i + kStages < n) fill(i + kStages);
  }
  // (after a timed-out wait: the copies that are on their way into the ring)
  if (!ok)
    for (int j = i - 1; j < min(n, i - 1 + kStages); ++j)
      mbar_wait(&full[j % kStages], (uint32_t)(j / kStages & 1));

  // ---- the warp's partial result, over its own ring
  float* part = reinterpret_cast<float*>(ring);  // [kRows][D], then m and l of each row
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float sum = l[half];
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    const int r = half * 8 + lane / 4;
#pragma unroll
    for (int d = 0; d < ND; ++d)
      *reinterpret_cast<float2*>(part + r * D + d * 8 + 2 * (lane & 3)) =
          make_float2(o[d][2 * half], o[d][2 * half + 1]);
    if ((lane & 3) == 0) {
      part[kRows * D + 2 * r] = m_use[half];
      part[kRows * D + 2 * r + 1] = sum;
    }
  }
  cluster.sync();

  // ---- join: the CTAs share the rows of all heads, four values a thread, and where
  // there are more threads than that several share a row's parts
  constexpr int kVec = D / 4;
  const int work = rows * hs * kVec, parts = ranks * slices;
  int lanes = 1;
  while (lanes < 16 && lanes < parts && work * lanes * 2 <= ranks * kThreads) lanes *= 2;
  const int my_part = lane & (lanes - 1);
#pragma unroll 1
  for (int w0 = rank * kThreads + warp * 32; w0 < work * lanes; w0 += ranks * kThreads) {
    const int w = min((w0 + lane) / lanes, work - 1);
    const int rh = w / kVec, c = w - rh * kVec;
    const int r = rh / hs, hh = rh - r * hs;
    float m = neg_inf(), sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // a part without a seen key counts for nothing; a NaN in one without any number
    // reaches the result
    auto add = [&](float mi, float li, float4 y) {
      const float top = fmaxf(m, mi);
      const float a = m == top ? 1.f : ex2(m - top), x = mi == top ? 1.f : ex2(mi - top);
      sum = fmaf(sum, a, x * li);
      acc.x = fmaf(acc.x, a, x * y.x);
      acc.y = fmaf(acc.y, a, x * y.y);
      acc.z = fmaf(acc.z, a, x * y.z);
      acc.w = fmaf(acc.w, a, x * y.w);
      m = top;
    };
#pragma unroll 2
    for (int i = my_part; i < parts; i += lanes) {
      const int cta = i / slices, wp = (i - cta * slices) * hs + hh;
      const float* f = cluster.map_shared_rank(
          reinterpret_cast<float*>(smem + wp * kStages * kStageBytes), cta);
      const float2 ml = *reinterpret_cast<const float2*>(f + kRows * D + 2 * r);
      const float4 y = *reinterpret_cast<const float4*>(f + r * D + 4 * c);
      if (ml.y != 0.f) add(ml.x, ml.y, y);
    }
#pragma unroll 1
    for (int o = 1; o < lanes; o <<= 1) {
      const float mi = __shfl_xor_sync(0xffffffffu, m, o), li = __shfl_xor_sync(0xffffffffu, sum, o);
      const float4 y = make_float4(
          __shfl_xor_sync(0xffffffffu, acc.x, o), __shfl_xor_sync(0xffffffffu, acc.y, o),
          __shfl_xor_sync(0xffffffffu, acc.z, o), __shfl_xor_sync(0xffffffffu, acc.w, o));
      if (li != 0.f) add(mi, li, y);
    }
    if (my_part != 0 || (w0 + lane) / lanes >= work) continue;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int at = r / p.G, g = r - at * p.G;
    const int head = (h - warp % hs + hh) * p.G + g;
    uint2 u;
    u.x = E::from_f2(acc.x * inv, acc.y * inv);
    u.y = E::from_f2(acc.z * inv, acc.w * inv);
    T* dst = reinterpret_cast<T*>(p.out) + ((int64_t)(e.q0 + at) * p.Hq + head) * D + 4 * c;
    *reinterpret_cast<uint2*>(dst) = u;
    if (c == 0 && p.lse != nullptr)
      p.lse[(int64_t)head * p.total_q + e.q0 + at] =
          sum == 0.f ? neg_inf() : (m + log2f(sum)) * kLn2;
  }
  cluster.sync();  // no CTA leaves while its parts are read
}

template <int D, typename T>
cudaError_t launch_t(const CrossParams& p, const CUtensorMap& tmk, const CUtensorMap& tmv,
                     cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  static std::atomic<int> resident[64][kClusterLimit + 1];  // by device and size; 0: not known
  constexpr int smem = kWarps * kStages * kStageBytes + 1024;
  const cudaError_t e =
      allow_shared(reinterpret_cast<const void*>(cross_kernel<D, T>), smem, &allowed);
  if (e != cudaSuccess) return e;
  int hs = kWarps;
  while (p.Hkv % hs != 0) hs /= 2;
  const long long items = (long long)p.B * (p.Hkv / hs);
  if (items > 0x7fffffffll / kMaxCluster) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attrs[2] = {};
  cudaLaunchAttribute& at = attrs[0];
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  overlap_launch(&attrs[1]);
  cfg.attrs = attrs;
  cfg.numAttrs = 1;
  // As many CTAs as are resident together, with a tile a warp at least (two: 6.9 us
  // instead of 6.2 for 200 keys; no more than 1.5 an SM: 64 entries of one row 153 us
  // instead of 162, but 32 of five rows 27.7 instead of 23.6).  Twice as many where a
  // warp has kLong tiles even so, for entries of unlike lengths (one and two rounds: 64
  // entries of 100 to 1500 keys, 16 heads of 64, 47 tiles a warp, 48 and 40 us; 64 of
  // 100 to 4096 keys, 8 heads of 128, 99 and 93; 32 of 1500 keys, 16 tiles, 35 and 39).
  constexpr int kLong = 32;
  const int tiles = (p.max_k + cross_narrow_box(D) - 1) / cross_narrow_box(D);
  const int slices = kWarps / hs;
  int most = tiles / slices, ctas = 1;
  most = most < 1 ? 1 : most < kMaxCluster ? most : kMaxCluster;
  for (int rounds = 1; rounds <= 2; ++rounds) {
    for (ctas = most; ctas > 1; --ctas) {
      cfg.gridDim = dim3((unsigned)ctas);
      at.val.clusterDim.x = (unsigned)ctas;
      const int held = resident_clusters(cross_kernel<D, T>, cfg, ctas, resident);
      if (items <= (long long)rounds * held) break;
    }
    if (tiles / (ctas * slices) < kLong) break;
  }
  cfg.gridDim = dim3((unsigned)(items * ctas));
  at.val.clusterDim.x = (unsigned)ctas;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, cross_kernel<D, T>, p, hs, tmk, tmv);
}

}  // namespace

cudaError_t launch_cross_narrow(const CrossParams& p, const CUtensorMap& tmk,
                                const CUtensorMap& tmv, int D, int dtype, cudaStream_t st) {
  if (D == 64)
    return dtype == PA_F16 ? launch_t<64, __half>(p, tmk, tmv, st)
                           : launch_t<64, __nv_bfloat16>(p, tmk, tmv, st);
  return dtype == PA_F16 ? launch_t<128, __half>(p, tmk, tmv, st)
                         : launch_t<128, __nv_bfloat16>(p, tmk, tmv, st);
}

}  // namespace pa

using namespace pa;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The strides of an axis with one place do not matter.
bool fix_strides(int64_t* st, int64_t* sh, int64_t rows, int heads, int D) {
  if (heads == 1) *sh = D;
  if (rows <= 1) *st = (int64_t)heads * (*sh > D ? *sh : D);
  return *st > 0 && *sh > 0 && *st % 8 == 0 && *sh % 8 == 0;
}

// More rows of a kv head than this run on tcgen05, whose tiles hold 128.  Here and
// there: 5 rows, head dim 64, 27 and 55 us; with two tiles of 16 rows 24 rows 43 and
// 41 us, with three 16 to 40 rows 51 and 26 us; 32 rows of head dim 128 190 and 176.
constexpr int kNarrowRows = 16;
bool is_wide(int total_q, int max_seqlen_q, int G) {
  const long long rows = (long long)(max_seqlen_q < total_q ? max_seqlen_q : total_q) * G;
  return rows > kNarrowRows;
}

}  // namespace

extern "C" PA_API size_t pa_fwd_cross_workspace_size(int total_q, int max_seqlen_q, int Hq, int Hkv,
                                                     int D) {
  if (total_q <= 0 || max_seqlen_q <= 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv != 0 ||
      (D != 64 && D != 128))
    return 0;
  return is_wide(total_q, max_seqlen_q, Hq / Hkv) ? cross_wide_workspace(D) : 0;
}

extern "C" PA_API int pa_fwd_cross(const void* q, int64_t q_st, int64_t q_sh, const void* k,
                                   int64_t k_st, int64_t k_sh, const void* v, int64_t v_st,
                                   int64_t v_sh, const int32_t* cu_seqlens_q,
                                   const int32_t* cu_seqlens_k, const int32_t* seqlens_k,
                                   const uint8_t* key_mask, int B, int total_q, int total_k,
                                   int max_seqlen_q, int max_seqlen_k, int Hq, int Hkv, int D,
                                   float scale, void* out, float* lse, void* workspace,
                                   size_t workspace_bytes, int32_t* err_word, int dtype,
                                   pa_stream_t stream) {
  if (dtype != PA_F16 && dtype != PA_BF16) return set_error(PA_ERR_UNSUPPORTED, "dtype %d", dtype);
  if (D != 64 && D != 128) return set_error(PA_ERR_UNSUPPORTED, "head_dim %d (64 or 128)", D);
  if (Hq < 1 || Hkv < 1) return set_error(PA_ERR_INVALID_ARG, "head counts must be >= 1");
  if (Hq % Hkv != 0)
    return set_error(PA_ERR_UNSUPPORTED, "Hq %d not a multiple of Hkv %d", Hq, Hkv);
  if (B < 0 || total_q < 0 || total_k < 0 || max_seqlen_q < 0 || max_seqlen_k < 0)
    return set_error(PA_ERR_INVALID_ARG, "negative size");
  if (!(scale > 0.f) || !std::isfinite(scale * kLog2e))
    return set_error(PA_ERR_INVALID_ARG, "scale must be positive, and finite times log2(e)");
  if (B == 0 || total_q == 0 || max_seqlen_q == 0) return PA_OK;
  if (q == nullptr || cu_seqlens_q == nullptr || cu_seqlens_k == nullptr || out == nullptr)
    return set_error(PA_ERR_INVALID_ARG, "q, cu_seqlens_q, cu_seqlens_k and out must be non-NULL");
  if (total_k > 0 && (k == nullptr || v == nullptr))
    return set_error(PA_ERR_INVALID_ARG, "k and v must be non-NULL");
  if (!aligned16(q) || !aligned16(out) || !aligned16(k) || !aligned16(v))
    return set_error(PA_ERR_INVALID_ARG, "q, k, v and out must be 16-byte aligned");
  if (!fix_strides(&q_st, &q_sh, total_q, Hq, D) || !fix_strides(&k_st, &k_sh, total_k, Hkv, D) ||
      !fix_strides(&v_st, &v_sh, total_k, Hkv, D))
    return set_error(PA_ERR_INVALID_ARG, "strides must be positive multiples of 8 elements");
  // (places up to a tile behind the last row or key still fit in 32 bits)
  if (total_q > 0x7fffffff - 4096 || total_k > 0x7fffffff - 4096)
    return set_error(PA_ERR_UNSUPPORTED, "more than 2^31 - 4097 rows or keys");
  const int G = Hq / Hkv;
  const int max_q = max_seqlen_q < total_q ? max_seqlen_q : total_q;
  const int max_k = max_seqlen_k < total_k ? max_seqlen_k : total_k;
  const long long tiles = ((long long)max_q * G + 15) / 16;
  if ((long long)B * Hkv * tiles > (1 << 26))
    return set_error(PA_ERR_UNSUPPORTED, "more than 2^26 tiles of 16 rows per kv head");
  const bool wide = is_wide(total_q, max_seqlen_q, G);
  // (the most heads that fit in a tile of 128 rows and divide G)
  int heads = G < 128 ? G : 128;
  while (wide && G % heads != 0) --heads;
  if (wide && (workspace == nullptr || workspace_bytes < cross_wide_workspace(D) ||
               (reinterpret_cast<uintptr_t>(workspace) & 255) != 0))
    return set_error(PA_ERR_WORKSPACE, "workspace of %zu bytes, 256-byte aligned, is needed",
                     cross_wide_workspace(D));
  if (wide) {  // (tiles are counted in 32 bits)
    const long long pair = 2 * (128 / heads);
    if ((long long)B * Hkv * (G / heads) * ((max_q + pair - 1) / pair) >
        (1 << 30) / (max_k / 128 + 1))
      return set_error(PA_ERR_UNSUPPORTED, "more than 2^30 tiles of 256 rows per kv head by 128 keys");
  }
  CrossParams p{};
  p.q = q;
  p.q_st = q_st;
  p.q_sh = q_sh;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.lens_k = seqlens_k;
  p.key_mask = key_mask;
  p.B = B;
  p.total_q = total_q;
  p.total_k = total_k;
  p.max_q = max_q;
  p.max_k = max_k;
  p.Hq = Hq;
  p.kv_split = wide ? G / heads : 1;
  p.Hkv = Hkv * p.kv_split;
  p.G = G / p.kv_split;
  p.scale_log2 = scale * kLog2e;
  p.out = out;
  p.lse = lse;
  p.err = err_word;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // (without keys nothing is read through the maps; they still need an address)
  const void* kb = total_k > 0 ? k : q;
  const void* vb = total_k > 0 ? v : q;
  const int64_t rows = total_k > 0 ? total_k : 1;
  const int box = wide ? 128 : cross_narrow_box(D);
  // A row of one head is 128 or 256 bytes.  The few-row kernel's warps read neighbouring
  // heads, so 256 suit it at head dim 64, too (128: no difference); on tcgen05 the next
  // head is another CTA's or later (16 entries of 8192 keys 94 us with 256, 75 with 128).
  const int l2 = wide && D == 64 ? 128 : 256;
  CUtensorMap tmq, tmk, tmv;
  if (!encode_map(&tmk, kb, dtype, D, Hkv, rows, 1, k_sh, k_st, k_st, 64, 1, box, true, l2) ||
      !encode_map(&tmv, vb, dtype, D, Hkv, rows, 1, v_sh, v_st, v_st, 64, 1, box, true, l2) ||
      (wide && !encode_map(&tmq, q, dtype, D, Hq, total_q, 1, q_sh, q_st, q_st, 64, p.G, 128 / p.G,
                           true, 256)))
    return set_error(PA_ERR_CUDA, "the tensor maps of q, k and v could not be encoded");
  const cudaError_t e = wide ? launch_cross_wide(p, tmq, tmk, tmv, D, dtype, workspace, st)
                             : launch_cross_narrow(p, tmk, tmv, D, dtype, st);
  if (e != cudaSuccess) return set_error(PA_ERR_CUDA, "cross launch: %s", cudaGetErrorString(e));
  return PA_OK;
}
