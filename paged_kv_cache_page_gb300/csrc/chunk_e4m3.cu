// Attention of prompt chunks over a paged e4m3 cache on the 5th-generation
// tensor cores (sm_103a): sequences of more query rows per kv head than the
// warp-level kernel (attend_e4m3.cu) takes.
//
// Mathematics as there: both products in fp16 with fp32 accumulation, e4m3
// being exact in fp16.  The rows of a tile are packed over the heads of a kv
// head, row i G + g of a sequence, so that all 256 rows of a CTA's two tiles
// share every K and V tile and its conversion.
//
// Bound: the tensor cores and the exponentials, 4 D operations and one
// exponential a visible (row, key) pair.  Two chunks of 2048 rows a head on 4096
// keys (32 heads on 8, D = 128) run in 209 us, 985 TFLOP/s, 0.51 of the measured
// library product.  Of the 3500 cycles of a tile (256 rows, 128 keys) the MMAs
// are 2050; what fills the rest is the chain of one group -- scores, softmax (2500
// cycles beside the other group's and the converters), both products.  A
// segment's end, where the softmax warps write results, costs 7000 to 12000
// cycles, an eighth of the time.  Registers are what most steps ran into: a
// role that spills bytes on their way waits for them (converters, 17 rows a
// sequence: 420 against 320 us).  Warps:
//   0-7    softmax: one thread a row, group g = warp / 4 takes tile g
//   8-11   converters: K and V tiles in turn -- 16 bytes a load from the pages,
//          two fp16 chunks a store into the 128-byte-swizzled operand tile --
//          into a ring of fp16 tiles K0 V0 K1 V1 ...
//   12     issues O_g += P_g V (P_g from TMEM over S_g) and S_g = Q_g K^T
//   13-14  Q of the next segment (a bf16 row scaled by a power of two), into the
//          other of two buffers
// TMEM: S_0, S_1, O_0, O_1.  While one group's softmax runs, the tensor core
// works on the other group.
//
// Work: the streams (sequence, kv head, pair of tiles) laid end to end in
// 128-key tiles, as many as the pair's last row sees, and dealt to the CTAs in
// equal shares or in slots (below); split streams are joined by the CTA that
// finishes last.
#include <algorithm>
#include <type_traits>

#include "attend_e4m3.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

// MMAs and commits under a predicate: a branch around them would take the warp's
// operands out of the uniform registers.
__device__ __forceinline__ void mma_ss_if(uint32_t on, uint32_t d, uint64_t a, uint64_t b,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t on, uint32_t d, uint32_t a, uint64_t b,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t on, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(on)
      : "memory");
}

constexpr int kM = 128;          // rows of a query tile
constexpr int kN = 128;          // keys of a tile
constexpr int kUnits = kN / kPage;
constexpr int kWarpConv = 8, kWarpMma = 12;
constexpr int kThreads = 15 * 32;
// The limits of the dealing, with both sides (us): 24 whole prompts of 300 tokens
// 145 with a least share of 4 tiles, 200 with 16 (and 145 with 1); 8 whole prompts
// of 1000 tokens 226 with cuts moved over up to 4 tiles, 243 over none, 249 over 12.
constexpr int kMinShare = 4;     // tiles
constexpr int kSnap = 4;         // tiles that a cut moves to an end of its stream

template <int D>
struct Layout {
  static constexpr int kHalves = D / 64;          // 64-column slabs of a row
  static constexpr int kSlab = 128 * 128;         // 128 rows x 128 bytes
  static constexpr int kTile = kHalves * kSlab;   // a fp16 operand tile
  static constexpr int kRing = D == 128 ? 3 : 8;  // K and V tiles in the ring
  static constexpr int kOffQ = 0;                 // [2 buffers][2]
  static constexpr int kOffKV = 4 * kTile;
  static constexpr int kOffF = kOffKV + kRing * kTile;      // float [256] factor of a row's scores
  static constexpr int kOffNan = kOffF + kChunkRows * 4;    // int [kRing][4]
  static constexpr int kOffWalk = kOffNan + kRing * 16;     // Walk [4], the converters'
  static constexpr int kOffBar = kOffWalk + 4 * 72;
  // q_full, q_empty [2], f_empty; full, empty [kRing]; s_full, p_full, pv_done, o_free [2]
  static constexpr int kBars = 5 + 2 * kRing + 8;
  static constexpr int kOffMisc = kOffBar + kBars * 8;      // TMEM base, merge flag
  static constexpr int kOffSums = kOffKV;                   // long long [kThreads + 16]; int [B] from
                                                            // 16 kThreads on; prologue
  static constexpr int kBytes = kOffMisc + 16 + 1024;
  static_assert(kBytes <= 232448, "shared memory");
};

struct Stream {  // a sequence with rows of this kernel's, and its share of tiles
  SeqRows s;
  int rows;      // qlen * G, 0: not this kernel's
  int pairs;
};

__device__ __forceinline__ Stream load_stream(const AttendParams& p, int b, bool tell) {
  Stream x{seq_rows(p, b, tell), 0, 0};
  const long long rows = (long long)x.s.qlen * p.G;
  if (rows > p.small_rows) {
    x.rows = (int)rows;
    x.pairs = (x.rows + kChunkRows - 1) / kChunkRows;
  }
  return x;
}

// Keys that row `row` of the sequence sees.
__device__ __forceinline__ int seen(const AttendParams& p, const Stream& x, int row) {
  return p.causal ? max(0, min(x.s.lk, row / p.G + x.s.lk - x.s.qlen + 1)) : x.s.lk;
}
// Key tiles of rows [row0, row0 + n) of the sequence.
__device__ __forceinline__ int tiles_of(const AttendParams& p, const Stream& x, int row0, int n) {
  const int last = min(row0 + n, x.rows) - 1;
  return last < row0 ? 0 : (seen(p, x, last) + kN - 1) / kN;
}
__device__ __forceinline__ int pair_tiles(const AttendParams& p, const Stream& x, int pair) {
  return max(1, tiles_of(p, x, pair * kChunkRows, kChunkRows));
}
// Cost of pair `i`: its tiles or, where streams are cut into slots of at most
// `slot` tiles, the number of them.
__device__ __forceinline__ int cost_of(int tiles, int slot) {
  return slot > 0 ? (tiles - 1) / slot + 1 : tiles;
}

// A segment of a CTA's share: tiles [t0, t0 + n) of a stream.
struct Walk {
  int b, h, pair, t0, n, all;  // all: tiles of the stream
  int slot;
  long long left;              // cost of the share from t0 on
  long long begin;             // cost of the streams in front
  Stream x;

  __device__ __forceinline__ int rows0() const { return pair * kChunkRows; }
  // End of the tiles that group g has work in.
  __device__ __forceinline__ int group_end(const AttendParams& p, int g) const {
    return min(t0 + n, tiles_of(p, x, rows0() + g * kM, kM));
  }
  // The stream behind this one.
  __device__ __forceinline__ void next_stream(const AttendParams& p) {
    begin += cost_of(all, slot);
    t0 = 0;
    if (++pair == x.pairs) {
      pair = 0;
      if (++h == p.Hkv) {
        h = 0;
        do {
          if (++b >= p.B) {  // (lengths that change under the launch)
            left = 0;
            return;
          }
          x = load_stream(p, b, false);
        } while (x.rows == 0);
      }
    }
    all = pair_tiles(p, x, pair);
  }
  __device__ __forceinline__ void next(const AttendParams& p) {
    left -= slot > 0 ? 1 : n;
    n = 0;
    if (left <= 0) return;
    next_stream(p);
    n = (int)min((long long)all, left);
  }
};

static_assert(sizeof(Walk) <= 72 && sizeof(Walk) % 8 == 0, "kOffWalk");

// Scales the first `cols` columns of fp16 probabilities in TMEM by a power of
// two a lane: exactly, but for what leaves fp16's normal range (2^-24 of the
// row's largest probability).  In two factors, for one below fp16's range would be
// zero where the probability, up to 2^15, is not.
__device__ __noinline__ void scale_p(uint32_t t, int cols, float by) {
  const float first = fmaxf(by, 0x1p-14f);
  const __half2 h0 = __float2half2_rn(first), h1 = __float2half2_rn(fminf(by * 0x1p14f, 1.f));
  tc::tmem_wait_st();
#pragma unroll 1
  for (int c = 0; c < cols; c += 16) {
    float v[16];
    uint32_t w[16];
    tc::tmem_ld16(t + c, v);
    tc::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t u = __float_as_uint(v[i]);
      const __half2 x = __hmul2(__hmul2(*reinterpret_cast<const __half2*>(&u), h0), h1);
      w[i] = *reinterpret_cast<const uint32_t*>(&x);
    }
    tc::tmem_st16u(t + c, w);
  }
  tc::tmem_wait_st();
}

// Adds the columns in which one of keys [key0, key1) of the sequence has a NaN
// in V (one bit a column).
template <int D>
__device__ __noinline__ void nan_columns(const AttendParams& p, int b, int h, int key0, int key1,
                                         uint32_t (&nans)[D / 32]) {
  for (int key = key0; key < key1; ++key) {
    const int unit = key / kPage;
    int page = __ldg(p.block_table + (int64_t)b * p.bt_stride + (unit >> p.page_shift));
    if (page < 0 || page >= p.num_pages) page = 0;
    const int row = (unit & ((1 << p.page_shift) - 1)) * kPage + key % kPage;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.v_cache + page * p.v_sb +
                                                            (int64_t)row * p.v_st + h * p.v_sh);
    for (int i = 0; i < D / 32; ++i)
      for (int e = 0; e < 8; ++e)  // bits 7, 15, 23, 31 to bits 0 to 3
        nans[i] |= ((((nan_bytes(__ldg(src + i * 8 + e)) >> 7) * 0x00204081u) >> 21) & 0xfu)
                   << (4 * e);
  }
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n)
               : "memory");
}

// As load16, past L1: what another CTA has written.
__device__ __forceinline__ float4 load16_l2(const void* src) {
  float4 x;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "l"(src)
               : "memory");
  return x;
}

// Two fp32 values at a time.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
  return x;
}
__device__ __forceinline__ float2 halves(uint64_t x) {
  float2 y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(x));
  return y;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t x;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(x) : "l"(a), "l"(b), "l"(c));
  return x;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t x;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(a), "l"(b));
  return x;
}

// Ties 32 values of an asynchronous TMEM load to the wait in front of it, so
// that nothing computed from them moves ahead of the wait.
__device__ __forceinline__ void arrived(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(v[i]));
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__
                                                                AttendParams p) {
  using L = Layout<D>;
  using E = Elem<T>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = smem + L::kOffQ;
  uint8_t* sKV = smem + L::kOffKV;
  float* sF = reinterpret_cast<float*>(smem + L::kOffF);
  int* sNan = reinterpret_cast<int*>(smem + L::kOffNan);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* q_full = bars;        // [2]
  uint64_t* q_empty = bars + 2;   // [2]
  uint64_t* f_empty = bars + 4;   // the score factors have been read
  uint64_t* full = bars + 5;
  uint64_t* empty = full + L::kRing;
  uint64_t* s_full = empty + L::kRing;
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 2;
  uint64_t* o_free = pv_done + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  int* sFlag = reinterpret_cast<int*>(smem + L::kOffMisc) + 1;
  long long* sSums = reinterpret_cast<long long*>(smem + L::kOffSums);
  int* sStreams = reinterpret_cast<int*>(smem + L::kOffF);  // [warps], prologue

  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 8);
      mbar_init(&q_empty[i], 9);  // the MMAs' reads, and the results staged there
    }
    mbar_init(f_empty, 8);
    for (int i = 0; i < L::kRing; ++i) {
      mbar_init(&full[i], 4);
      mbar_init(&empty[i], 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&s_full[g], 1);
      mbar_init(&p_full[g], 4);
      mbar_init(&pv_done[g], 1);
      mbar_init(&o_free[g], 4);
    }
    fence_mbar_init();
  }

  // ---- the CTA's share
  // A pass over the batch finds each sequence's cost, a warp a sequence, a lane a
  // pair, and its running sums, a thread kPer sequences.  The first pass counts
  // tiles.  Fewer streams than CTAs are then cut into slots, one a CTA, of a
  // length that half a slot a stream less fills the CTAs with (second pass) or,
  // where there are more of those than CTAs, that always does (third).
  int* sCost = reinterpret_cast<int*>(smem + L::kOffSums) + 4 * kThreads;  // [B]
  const int per = (p.B + kThreads - 1) / kThreads, ctas = (int)gridDim.x;
  long long total = 0, tiles = 0;
  int slot = 0, streams = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    int mine = 0;
    for (int b = warp; b < p.B; b += kThreads / 32) {
      const Stream x = load_stream(p, b, false);
      int cost = 0;
      for (int i = lane; i < x.pairs; i += 32) cost += cost_of(pair_tiles(p, x, i), slot);
      cost = __reduce_add_sync(0xffffffffu, cost);
      if (lane == 0) sCost[b] = cost;
      mine += x.pairs;
    }
    if (lane == 0) sStreams[warp] = mine;
    __syncthreads();
    long long incl = 0;
    for (int i = 0; i < per; ++i)
      if (tid * per + i < p.B) incl += (long long)sCost[tid * per + i] * p.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sSums[kThreads + warp] = incl;
    __syncthreads();
    total = 0;
    streams = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      const long long x = sSums[kThreads + w];
      if (w < warp) incl += x;
      total += x;
      streams += sStreams[w];
    }
    sSums[tid] = incl;
    __syncthreads();
    const long long all_streams = (long long)streams * p.Hkv;
    if (pass == 0) tiles = total;
    if (all_streams >= ctas || (pass > 0 && total <= ctas)) break;
    const float room = pass == 0 ? (float)ctas - 0.5f * (float)all_streams
                                 : (float)ctas - (float)all_streams;
    slot = (int)((float)tiles / room) + 2;
  }
  // Otherwise equal shares of the tiles.  A cut at most kSnap tiles from an end of
  // its stream moves there: a segment costs about as much as that many tiles.
  const long long share =
      slot > 0 ? 1 : max(quotient(total + ctas - 1, ctas), (long long)kMinShare);
  if (share * blockIdx.x >= total) return;
  Walk at{};
  at.slot = slot;
  long long end = 0;
#pragma unroll 1
  for (int side = 1; side >= 0; --side) {  // the end of the share, then its begin
    const long long cut = share * (blockIdx.x + side);
    if (side == 1 && (slot > 0 || cut >= total)) {
      end = min(cut, total);
      continue;
    }
    int lo = 0;
    for (int step = 256; step > 0; step >>= 1)
      if (lo + step <= kThreads && sSums[lo + step - 1] <= cut) lo += step;
    at.begin = lo > 0 ? sSums[lo - 1] : 0;
    at.b = lo * per;
    while (at.b + 1 < p.B && cut - at.begin >= (long long)sCost[at.b] * p.Hkv)
      at.begin += (long long)sCost[at.b++] * p.Hkv;
    at.x = load_stream(p, at.b, false);
    const int head = max(sCost[at.b], 1);
    const long long off = cut - at.begin;
    at.h = (int)quotient(off, head);
    at.begin += (long long)at.h * head;
    int rest = (int)(off - (long long)at.h * head);
    // the pair: 32 a step, by a scan over the lanes
    at.pair = 0;
#pragma unroll 1
    for (int i0 = 0;; i0 += 32) {
      const int i = i0 + lane;
      const int cost = i < at.x.pairs ? cost_of(pair_tiles(p, at.x, i), slot) : 0;
      int sum = cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, sum > rest);
      if (past == 0 && i0 + 32 < at.x.pairs) {
        const int step = __shfl_sync(0xffffffffu, sum, 31);
        rest -= step;
        at.begin += step;
        continue;
      }
      const int l = past != 0 ? __ffs(past) - 1 : 0;
      const int before = __shfl_sync(0xffffffffu, sum - cost, l);
      rest -= before;
      at.begin += before;
      at.pair = i0 + l;
      break;
    }
    at.all = pair_tiles(p, at.x, at.pair);
    at.t0 = rest;
    if (slot > 0) {
      const int chunk = (at.all - 1) / cost_of(at.all, slot) + 1;
      at.t0 = rest * chunk;
      at.n = min(chunk, at.all - at.t0);
      at.left = 1;
    } else {
      if (blockIdx.x + side > 0) {
        if (at.t0 <= kSnap) at.t0 = 0;
        else if (at.all - at.t0 <= kSnap) at.next_stream(p);
      }
      if (side == 1) {
        end = at.begin + at.t0;
      } else {
        at.left = end - (at.begin + at.t0);
        at.n = (int)min((long long)(at.all - at.t0), at.left);
      }
    }
  }
  if (at.left <= 0) return;
  if (warp == kWarpMma) {
    tc::tmem_alloc(tslot, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();  // (and sSums has been read)
  tc::fence_after_sync();
  const uint32_t tbase = *tslot;
  auto tS = [&](int g) { return tbase + (uint32_t)(g * 128); };
  auto tO = [&](int g) { return tbase + 256u + (uint32_t)(g * D); };
  bool failed = false;
  auto wait = [&](uint64_t* bar, uint32_t par, int where) {
    if (!failed && !mbar_wait(bar, par)) {
      report(p.err, PA_DEVERR_TIMEOUT, -1, where);
      failed = true;
    }
  };

  // Q of the pair of segment `w` into buffer `buf`, by `threads` threads of
  // whole warps, 16 (D = 64: 8) lanes a row: copied to its place by cp.async,
  // then turned in place where it is not yet as the MMAs read it -- a bf16 row
  // is scaled by a power of two to a largest magnitude in [1, 2); a negative
  // scale of K turns the signs, so that no score factor is negative.  Four rows
  // a step: one at a time, two warps needed 33000 cycles for a segment's rows,
  // more than the tiles of a short prompt (24 of 300 tokens 144 us, 104 with
  // four); unrolled whole, code that runs once comes from far away, and the
  // first segment's rows took 28000 cycles, waiting for instructions.
  auto stage_q = [&](const Walk& w, int buf, int i, int threads) {
    constexpr int kLanes = D / 8;
    const int qc = i % kLanes, step = threads / kLanes;
    const uint32_t flip =
        p.k_scale != nullptr && __ldg(p.k_scale + w.h) < 0.f ? 0x80008000u : 0u;
    uint8_t* tile = sQ + buf * 2 * L::kTile + (qc >> 3) * L::kSlab;
    auto place = [&](int r) {
      const int rt = r & 127;
      return tile + (r >> 7) * L::kTile + rt * 128 + (((qc & 7) ^ (rt & 7)) << 4);
    };
    const T* base = reinterpret_cast<const T*>(p.q) + (int64_t)w.x.s.q0 * p.q_st +
                    (int64_t)(w.h * p.G) * p.q_sh + qc * 8;
    // row = token * G + head: divided once, then carried on
    int token = (w.rows0() + i / kLanes) / p.G, head = (w.rows0() + i / kLanes) % p.G;
    const int step_t = step / p.G, step_h = step % p.G;
#pragma unroll 4
    for (int r = i / kLanes; r < kChunkRows; r += step) {
      const bool live = w.rows0() + r < w.x.rows;
      const T* src = live ? base + (int64_t)token * p.q_st + (int64_t)head * p.q_sh : base;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(place(r))),
                   "l"(src), "r"(live ? 16 : 0)
                   : "memory");
      token += step_t;
      head += step_h;
      if (head >= p.G) {
        head -= p.G;
        ++token;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    constexpr bool kTurn = !std::is_same<T, __half>::value;
    if (kTurn || flip != 0) {
      constexpr int kAtOnce = 4;  // rows: their loads and reductions side by side
#pragma unroll 1
      for (int r = i / kLanes; r < kChunkRows; r += kAtOnce * step) {
        uint4 x[kAtOnce];
        float f[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          x[j] = *reinterpret_cast<const uint4*>(place(r + j * step));
          f[j] = 1.f;
        }
        if constexpr (kTurn) {
          uint32_t top[kAtOnce];
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            const uint32_t u[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
            top[j] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              top[j] = max(top[j], max((u[e] & 0x7fffu) << 16, u[e] & 0x7fff0000u));
          }
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1)
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
              top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            const int ex = (int)(top[j] >> 23);
            const bool turn = ex > 0 && ex < 255;
            const int by = min(ex, 253);
            const float down = turn ? __uint_as_float((uint32_t)(254 - by) << 23) : 1.f;
            if (turn) f[j] = __uint_as_float((uint32_t)by << 23);
            uint32_t u[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 y = E::to_f2(u[e]);
              u[e] = Elem<__half>::from_f2(y.x * down, y.y * down);
            }
            x[j] = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          *reinterpret_cast<uint4*>(place(r + j * step)) =
              make_uint4(x[j].x ^ flip, x[j].y ^ flip, x[j].z ^ flip, x[j].w ^ flip);
          if (qc == 0) sF[r + j * step] = f[j];
        }
      }
    } else if (qc == 0) {
      for (int r = i / kLanes; r < kChunkRows; r += step) sF[r] = 1.f;
    }
    fence_proxy_async_smem();
    __syncwarp();
  };

  if (warp == kWarpMma) {
    // ======================= MMA issuer =======================
    // Per tile and group: O_g += P_g V, then S_g of the next tile.  One thread's
    // MMAs run in the order it issues them, so S_g may follow the product that
    // reads P_g from the same columns without a wait.
    const uint32_t id_s = tc::idesc_f16(kM, kN, false, false);
    const uint32_t id_o = tc::idesc_f16(kM, D, false, true);
    // Descriptors move in their low words alone (addresses stay below 2^18), and
    // the high words are constants: the issuing thread's own instructions are
    // what slows a stream of N = 128 MMAs.
    const uint64_t d16 = tc::smem_desc(0, 16, 1024), dslab = tc::smem_desc(0, L::kSlab, 1024);
    const uint32_t qlo = (uint32_t)d16 + (smem_u32(sQ) >> 4), klo = (uint32_t)d16 + (smem_u32(sKV) >> 4);
    const uint32_t vlo = (uint32_t)dslab + (smem_u32(sKV) >> 4);
    auto desc = [](uint64_t base, uint32_t lo) {
      uint64_t d;
      asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"((uint32_t)(base >> 32)));
      return d;
    };
    // The warp issues as one, an elected thread's predicate on, and every operand
    // is broadcast, which lets the compiler hold it in uniform registers: branching
    // to lane 0, a tile's 32 MMAs took 125 cycles each to issue, so they take 78
    // (64 is the tensor core's own rate): two chunks of 2048 on 4096 keys 255 -> 229
    // us.
    auto uni = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
    uint32_t on;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(on));
    const uint32_t tb = uni(tbase);
    int k = 0, a = 0, n0 = 0, n1 = 0, m0 = 0, m1 = 0;
    auto scores = [&](int g, int s) {
      const uint32_t q0 = uni(qlo + (uint32_t)((((a & 1) * 2 + g) * L::kTile) >> 4));
      const uint32_t k0 = uni(klo + (uint32_t)((s * L::kTile) >> 4));
      const uint32_t ts = uni(tb + g * 128);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * L::kSlab + (kk & 3) * 32) >> 4;
        mma_ss_if(on, ts, desc(d16, q0 + off), desc(d16, k0 + off), id_s, kk > 0);
      }
      commit_if(on, &s_full[g]);
      __syncwarp();
    };
    auto release = [&](uint64_t* bar) {
      commit_if(on, bar);
      __syncwarp();
    };
    for (; at.left > 0; at.next(p), ++a) {
      const int end0 = at.group_end(p, 0), end1 = at.group_end(p, 1), end = at.t0 + at.n;
      wait(&q_full[a & 1], (uint32_t)((a >> 1) & 1), 40);
      wait(&full[k % L::kRing], (uint32_t)((k / L::kRing) & 1), 41);
      tc::fence_after_sync();
      if (at.t0 < end0) scores(0, k % L::kRing);
      if (at.t0 < end1) scores(1, k % L::kRing);
      release(&empty[k % L::kRing]);
      for (int t = at.t0; t < end; ++t, k += 2) {
        const int v = k + 1, kn = k + 2;  // places of V of this tile and K of the next
        const int sv = v % L::kRing, sk = kn % L::kRing;
        wait(&full[sv], (uint32_t)((v / L::kRing) & 1), 50);
        bool next_k = false;  // K of the next tile has been waited for
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
          const int gend = g ? end1 : end0;
          if (t < gend) {
            const int n = g ? n1 : n0, m = g ? m1 : m0;
            wait(&p_full[g], (uint32_t)(n & 1), 51 + g);
            if (t == at.t0 && m >= 1) wait(&o_free[g], (uint32_t)((m - 1) & 1), 53 + g);
            tc::fence_after_sync();
            const uint32_t v0 = uni(vlo + (uint32_t)((sv * L::kTile) >> 4));
            const uint32_t ts = uni(tb + g * 128), to = uni(tb + 256 + g * D);
            const uint32_t more = uni(t > at.t0);
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk)
              mma_ts_if(on, to, ts + kk * 8, desc(dslab, v0 + (kk * 2048 >> 4)), id_o,
                        kk > 0 ? 1u : more);
            commit_if(on, &pv_done[g]);
            __syncwarp();
            if (g) ++n1;
            else ++n0;
            if (t + 1 < gend) {
              if (!next_k) {
                wait(&full[sk], (uint32_t)((kn / L::kRing) & 1), 41);
                tc::fence_after_sync();
                next_k = true;
              }
              scores(g, sk);
            }
          }
        }
        release(&empty[sv]);
        if (t + 1 < end) release(&empty[sk]);
      }
      release(&q_empty[a & 1]);
      if (end0 > at.t0) ++m0;
      if (end1 > at.t0) ++m1;
    }
  } else if (warp > kWarpMma) {
    // ======================= Q of the segments behind the first ===============
    // One segment ahead, into the buffer that the segment before has left.
    int a = 0;
    for (; at.left > 0; at.next(p), ++a) {
      if (a == 0) continue;  // the softmax warps, which have nothing to do yet
      if (a >= 2) wait(&q_empty[a & 1], (uint32_t)(((a >> 1) - 1) & 1), 10);
      wait(f_empty, (uint32_t)((a - 1) & 1), 11);
      stage_q(at, a & 1, tid - (kWarpMma + 1) * 32, 64);
      if (lane == 0) mbar_arrive_n(&q_full[a & 1], 4);
    }
    // nothing in flight may outlive the CTA: the last reads of either buffer
    for (int b = max(0, a - 2); b < a; ++b) wait(&q_empty[b & 1], (uint32_t)((b >> 1) & 1), 12);
  } else if (warp >= kWarpConv) {
    // ======================= converters =======================
    const int ct = tid - kWarpConv * 32;  // 0 .. 127
    constexpr int kChunks = D / 16;       // 16-byte chunks of a key
    constexpr int kRowsAt = 128 / kChunks;
    constexpr int kLoads = kN / kRowsAt;  // of a thread and tile
    // Chunk and key: eight lanes take four chunks of two neighbouring keys, whose
    // swizzled places cover every bank once.
    const int c = D == 128 ? (ct & 3) | ((ct >> 1) & 4) : ct & 3;
    const int r0 = D == 128 ? ((ct >> 2) & 1) | ((ct >> 4) << 1) : ct >> 2;
    int k = 0;
    // The position waits in shared memory: with it in registers the compiler
    // spills bytes that are on their way, which waits for them.
    Walk* parked = reinterpret_cast<Walk*>(smem + L::kOffWalk) + (warp - kWarpConv);
    while (at.left > 0) {
      const int t0 = at.t0, t1 = at.t0 + at.n;
      const int least = seen(p, at.x, at.rows0());  // keys that the pair's first row sees
      if (lane == 0) *parked = at;
      __syncwarp();
      const int32_t* trow = p.block_table + (int64_t)at.b * p.bt_stride;
      const int lk = at.x.s.lk;
      // Lane l finds unit `unit` + l of 32 units (four tiles): the table entry,
      // and later its place in either cache.  An entry outside the pool is
      // reported and read as page 0, as is what lies behind the last key.
      auto table = [&](int unit) {
        unit += lane;
        return unit * kPage < lk ? __ldg(trow + (unit >> p.page_shift)) : 0;
      };
      int64_t koff, voff;
      auto place = [&](int entry, int unit) {
        unit += lane;
        if (entry < 0 || entry >= p.num_pages) {
          if (ct < 32) report(p.err, PA_DEVERR_PAGE_OOB, parked->b, unit);
          entry = 0;
        }
        const int row = (unit & ((1 << p.page_shift) - 1)) * kPage;
        koff = entry * p.k_sb + row * p.k_st;
        voff = entry * p.v_sb + row * p.v_st;
      };
      const uint8_t* kbase = p.k_cache + (int64_t)at.h * p.k_sh + c * 16 + (r0 & 15) * p.k_st;
      const uint8_t* vbase = p.v_cache + (int64_t)at.h * p.v_sh + c * 16 + (r0 & 15) * p.v_st;
      // The thread's 16 bytes of each of its keys of tile t: loads without a
      // condition (rows behind the last key lie in its page or in page 0, and
      // are cleared before they are stored), so that all are in flight at once.
      auto load = [&](const uint8_t* base, int64_t off, int t, uint4 (&x)[kLoads]) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int unit = ((t - t0) & 3) * kUnits + (i * kRowsAt + r0) / kPage;
          x[i] = load16(base + __shfl_sync(0xffffffffu, (long long)off, unit));
        }
      };
      // Zeros at keys of tile t behind the last one.
      auto clear = [&](int t, uint4 (&x)[kLoads]) {
        if ((t + 1) * kN <= lk) return;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          if (t * kN + i * kRowsAt + r0 >= lk) x[i] = make_uint4(0, 0, 0, 0);
      };
      place(table(t0 * kUnits), t0 * kUnits);
      int nxt = t1 - t0 > 4 ? table((t0 + 4) * kUnits) : 0;
      uint4 xk[kLoads], xv[kLoads];
      load(kbase, koff, t0, xk);
      auto store = [&](uint8_t* tile, const uint4 (&x)[kLoads]) {
        uint8_t* slab = tile + (c >> 2) * L::kSlab;
        const int c0 = 2 * (c & 3);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int r = i * kRowsAt + r0;
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) f16x4_of(w[e], h[2 * e], h[2 * e + 1]);
          *reinterpret_cast<uint4*>(slab + r * 128 + ((c0 ^ (r & 7)) << 4)) =
              make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(slab + r * 128 + (((c0 + 1) ^ (r & 7)) << 4)) =
              make_uint4(h[4], h[5], h[6], h[7]);
        }
      };
      auto done = [&](int s) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      };
      for (int t = t0; t < t1; ++t) {
        // V of this tile and K of the next are on their way while K of this one
        // is converted
        load(vbase, voff, t, xv);
        int s = k % L::kRing;
        wait(&empty[s], (uint32_t)(((k / L::kRing) & 1) ^ 1), 20);
        clear(t, xk);
        store(sKV + s * L::kTile, xk);
        done(s);
        ++k;
        if (t + 1 < t1) {
          if (((t + 1 - t0) & 3) == 0) {
            place(nxt, (t + 1) * kUnits);
            if (t + 5 < t1) nxt = table((t + 5) * kUnits);
          }
          load(kbase, koff, t + 1, xk);
        }
        s = k % L::kRing;
        wait(&empty[s], (uint32_t)(((k / L::kRing) & 1) ^ 1), 21);
        clear(t, xv);
        if ((t + 1) * kN > least) {
          // Some row does not see all of the tile: a NaN in V is taken out of
          // the product (0 x NaN) and told to the rows, which put it into
          // their results if they see it.
          uint32_t bad = 0;
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&xv[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t hit = nan_bytes(w[e]);
              bad |= hit;
              w[e] &= ~((hit >> 7) * 0xffu);
            }
          }
          const bool any = __any_sync(0xffffffffu, bad != 0);
          if (lane == 0) sNan[s * 4 + warp - kWarpConv] = any ? 1 : 0;
        }
        store(sKV + s * L::kTile, xv);
        done(s);
        ++k;
      }
      __syncwarp();
      at = *parked;
      __syncwarp();
      at.next(p);
    }
    // nothing in flight may outlive the CTA: the last reads of the ring
    for (int i = 0; i < L::kRing; ++i, ++k)
      wait(&empty[k % L::kRing], (uint32_t)(((k / L::kRing) & 1) ^ 1), 22);
  } else {
    // ======================= softmax =======================
    const int g = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    int n = 0, a = 0, k = 1;  // k: the V tile's place in the ring
    for (; at.left > 0; ++a) {
      const int row = at.rows0() + g * kM + r;
      const bool valid = row < at.x.rows;
      const int qi = valid ? row / p.G : 0, h = at.h * p.G + (valid ? row % p.G : 0);
      const float ks = p.k_scale != nullptr ? __ldg(p.k_scale + at.h) : 1.f;
      const float vs = p.v_scale != nullptr ? __ldg(p.v_scale + at.h) : 1.f;
      if (a == 0) {
        stage_q(at, 0, tid, 256);
        if (lane == 0) mbar_arrive(&q_full[0]);
      }
      wait(&q_full[a & 1], (uint32_t)((a >> 1) & 1), 59);
      const float f = sF[g * kM + r] * (fabsf(ks) * p.scale_log2);
      __syncwarp();
      if (lane == 0) mbar_arrive(f_empty);
      const int sees = valid ? seen(p, at.x, row) : 0;
      const int least = seen(p, at.x, at.rows0());
      const int end = at.group_end(p, g);
      float m = neg_inf(), l = 0.f;
      uint32_t nans[D / 32];  // columns of the row that a NaN in V reaches
#pragma unroll
      for (int i = 0; i < D / 32; ++i) nans[i] = 0;
      for (int t = at.t0; t < end; ++t) {
        wait(&s_full[g], (uint32_t)(n & 1), 60 + g);
        tc::fence_after_sync();
        const uint32_t ts = tS(g) + lane_off;
        const int lim = sees - t * kN;  // keys [0, lim) of the tile are seen
        const bool whole = lim >= kN;
        // One pass over the row's scores, 32 at a time in a rolled loop: the
        // loads take 40 cycles, but unrolled over the tile the code of the
        // roles passes what the instruction caches hold, and every warp waits
        // for instructions.
        float v[32];
        uint64_t sum2[4] = {0, 0, 0, 0};  // four pairs of sums
        float alpha = 1.f;
        auto probabilities = [&](auto masked, int key0) {
          const int left = lim - key0;
          if constexpr (masked) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = i < left ? v[i] : neg_inf();
          }
          // The exponentials do not wait for the largest score: the chunk is done
          // again where it passes the reference by more than the slack.
          uint32_t pk[16];
          uint64_t more[4];
#pragma unroll 1
          for (;;) {
            const float neg_m = m == neg_inf() ? 0.f : -m;
            const uint64_t f2 = pair(f, f), m2 = pair(neg_m, neg_m);
            float top4[4];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 z = halves(fma2(pair(v[2 * e], v[2 * e + 1]), f2, m2));
              float e0 = ex2(z.x), e1 = ex2(z.y);
              if constexpr (masked) {  // (a factor of zero turns -inf into NaN)
                e0 = 2 * e < left ? e0 : 0.f;
                e1 = 2 * e + 1 < left ? e1 : 0.f;
              }
              more[e & 3] = e < 4 ? pair(e0, e1) : add2(more[e & 3], pair(e0, e1));
              top4[e & 3] = e < 4 ? fmaxf(v[2 * e], v[2 * e + 1]) : max3(top4[e & 3], v[2 * e], v[2 * e + 1]);
              pk[e] = Elem<__half>::from_f2(e0, e1);
            }
            const float top = max3(fmaxf(top4[0], top4[1]), top4[2], top4[3]) * f;
            const bool far = top > m + (kE4m3Shift + kE4m3Slack);
            if (!__any_sync(0xffffffffu, far)) break;
            // References are whole numbers, so what is scaled here is scaled
            // by powers of two: this tile's sums and probabilities so far, and
            // after the loop O.
            float by = 1.f;
            if (far) {
              const float to = ceilf(top) - kE4m3Shift;
              if (m != neg_inf()) by = ex2(m - to);
              m = to;
            }
            alpha *= by;
            l *= by;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 z = halves(sum2[i]);
              sum2[i] = pair(z.x * by, z.y * by);
            }
            scale_p(ts, key0 / 2, by);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) sum2[i] = add2(sum2[i], more[i]);
          // over the columns of scores that have been used
          tc::tmem_st16u(ts + key0 / 2, pk);
        };
        auto row = [&](auto masked) {
#pragma unroll 1
          for (int c = 0; c < kN; c += 32) {
            tc::tmem_ld32(ts + c, v);
            tc::tmem_wait_ld();
            arrived(v);
            probabilities(masked, c);
          }
        };
        if (__all_sync(0xffffffffu, whole))
          row(std::false_type{});
        else
          row(std::true_type{});
        const float2 sum = halves(add2(add2(sum2[0], sum2[1]), add2(sum2[2], sum2[3])));
        l += sum.x + sum.y;
        if (t > at.t0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // O_g is still once P V of the group's previous tile is done
          wait(&pv_done[g], (uint32_t)((n - 1) & 1), 62 + g);
          tc::fence_after_sync();
#pragma unroll 1
          for (int i = 0; i < D / 32; ++i) {
            float o[32];
            tc::tmem_ld32(tO(g) + lane_off + i * 32, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= alpha;
            tc::tmem_st32(tO(g) + lane_off + i * 32, o);
          }
        }
        if ((t + 1) * kN > least) {
          const int s = (k + 2 * (t - at.t0)) % L::kRing;
          wait(&full[s], (uint32_t)(((k + 2 * (t - at.t0)) / L::kRing) & 1), 66);
          const int4 bad = *reinterpret_cast<const int4*>(sNan + s * 4);
          if ((bad.x | bad.y | bad.z | bad.w) != 0) {
            nan_columns<D>(p, at.b, at.h, t * kN, min(sees, (t + 1) * kN), nans);
          }
          __syncwarp();
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[g]);
        ++n;
      }
      // ---- the segment's result
      const bool whole = at.n == at.all;
      const int slot = 2 * blockIdx.x + (at.t0 == 0 ? 1 : 0);
      const int64_t my_part = ((int64_t)slot * 2 + g) * kM;
      // Results leave by way of the segment's Q tile, which is not read any more:
      // a thread holds a row, and 32 rows a store instruction cost 32 cycles of
      // the memory pipe, two whole rows four.
      uint8_t* staged = sQ + ((a & 1) * 2 + g) * L::kTile;
      auto stage = [&](int c, uint4 x) {
        *reinterpret_cast<uint4*>(staged + r * (2 * D) + ((c ^ (r & 7)) << 4)) = x;
      };
      auto write_rows = [&]() {
        constexpr int kLanes = D / 8;
        const long long my_row = valid ? (long long)(at.x.s.q0 + qi) * p.Hq + h : -1;
        const int c = lane % kLanes;
        __syncwarp();
#pragma unroll 4
        for (int i = lane / kLanes; i < 32; i += 32 / kLanes) {
          const long long to = __shfl_sync(0xffffffffu, my_row, i);
          const int rt = quarter * 32 + i;
          const uint4 x = *reinterpret_cast<const uint4*>(staged + rt * (2 * D) + ((c ^ (rt & 7)) << 4));
          if (to >= 0) *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.out) + to * D + c * 8) = x;
        }
      };
      auto put_lse = [&](float ref, float sum) {
        if (p.lse != nullptr)
          p.lse[(int64_t)h * p.total_q + at.x.s.q0 + qi] =
              sum == 0.f ? neg_inf() : (ref + log2f(sum)) * kLn2;
      };
      const float nan = __int_as_float(0x7fffffff);
      if (end > at.t0) {
        wait(&pv_done[g], (uint32_t)((n - 1) & 1), 64 + g);
        tc::fence_after_sync();
        const float by = l == 0.f ? 0.f : vs / l;
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          float o[32];
          tc::tmem_ld32(tO(g) + lane_off + i * 32, o);
          tc::tmem_wait_ld();
          if (nans[i] != 0) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((nans[i] >> e) & 1) o[e] = nan;
          }
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              stage(i * 4 + e / 8,
                    make_uint4(E::from_f2(o[e] * by, o[e + 1] * by),
                               E::from_f2(o[e + 2] * by, o[e + 3] * by),
                               E::from_f2(o[e + 4] * by, o[e + 5] * by),
                               E::from_f2(o[e + 6] * by, o[e + 7] * by)));
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<float4*>(p.part_o + (my_part * (D / 4) + (i * 8 + e) * kM + r) * 4) =
                  make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[g]);
      } else if (whole) {
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) stage(c, make_uint4(0, 0, 0, 0));
      }
      if (whole) {
        write_rows();
        if (valid) put_lse(m, l);
      } else {
        p.part_ml[my_part + r] = make_float2(m, l);
        int cta0, cta1;
        if (at.slot > 0) {
          cta0 = (int)at.begin;
          cta1 = cta0 + cost_of(at.all, at.slot) - 1;
        } else {  // the cuts that were not moved to the stream's ends
          cta0 = (int)quotient(at.begin + kSnap, share);
          cta1 = (int)quotient(at.begin + at.all - kSnap - 1, share);
        }
        named_barrier(1, 256);  // the partial rows of the CTA before its arrival
        if (tid == 0) {
          __threadfence();
          *sFlag = arrive_last(p.words + cta0, launch_tag(), cta1 - cta0 + 1) ? 1 : 0;
          __threadfence();
        }
        named_barrier(1, 256);
        if (*sFlag) {
          // the first row of the stream's split n, of this thread's group
          auto from = [&](int cta) {
            return ((int64_t)(2 * cta + (cta == cta0 ? 1 : 0)) * 2 + g) * kM;
          };
          float ref = neg_inf(), sum = 0.f;
          for (int cta = cta0; cta <= cta1; ++cta)
            ref = fmaxf(ref, __ldcg(p.part_ml + from(cta) + r).x);
          // a row's part of a split: 0 where the group had no tile (O unset)
          auto weight = [&](float2 ml) {
            return ml.x == neg_inf() ? 0.f : ml.x == ref ? 1.f : ex2(ml.x - ref);
          };
          for (int cta = cta0; cta <= cta1; ++cta) {
            const float2 ml = __ldcg(p.part_ml + from(cta) + r);
            sum = fmaf(weight(ml), ml.y, sum);
          }
          const float by = sum == 0.f ? 0.f : vs / sum;
          constexpr int kPart = D / 16;  // 16-byte chunks of a quarter of the row
#pragma unroll 1
          for (int part = 0; part < 4; ++part) {
            float4 acc[kPart];
#pragma unroll
            for (int e = 0; e < kPart; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int cta = cta0; cta <= cta1; ++cta) {
              const int64_t at_row = from(cta);
              float4 y[kPart];
              const float2 ml = __ldcg(p.part_ml + at_row + r);
#pragma unroll
              for (int e = 0; e < kPart; ++e)
                y[e] = load16_l2(p.part_o + (at_row * (D / 4) + (part * kPart + e) * kM + r) * 4);
              // (an unset O is not used; one whose weight is 0 is, for it may hold NaN)
              if (ml.x == neg_inf()) continue;
              const float w = weight(ml);
#pragma unroll
              for (int e = 0; e < kPart; ++e) {
                acc[e].x = fmaf(w, y[e].x, acc[e].x);
                acc[e].y = fmaf(w, y[e].y, acc[e].y);
                acc[e].z = fmaf(w, y[e].z, acc[e].z);
                acc[e].w = fmaf(w, y[e].w, acc[e].w);
              }
            }
#pragma unroll
            for (int e = 0; e < kPart; e += 2)
              stage(part * (D / 32) + e / 2,
                    make_uint4(E::from_f2(acc[e].x * by, acc[e].y * by),
                               E::from_f2(acc[e].z * by, acc[e].w * by),
                               E::from_f2(acc[e + 1].x * by, acc[e + 1].y * by),
                               E::from_f2(acc[e + 1].z * by, acc[e + 1].w * by)));
          }
          write_rows();
          if (valid) put_lse(ref, sum);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[a & 1]);
      k += 2 * at.n;
      at.next(p);
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kWarpMma) tc::tmem_dealloc(tbase, 512);
}

template <int D, typename T>
cudaError_t launch(const AttendParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> devices{0};
  const cudaError_t e = allow_shared(reinterpret_cast<const void*>(chunk_kernel<D, T>),
                                     Layout<D>::kBytes, &devices);
  if (e != cudaSuccess) return e;
  chunk_kernel<D, T><<<(unsigned)num_sms(), kThreads, Layout<D>::kBytes, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunks_e4m3(const AttendParams& p, int D, int dtype, cudaStream_t st) {
  if (dtype == PA_F16) return D == 128 ? launch<128, __half>(p, st) : launch<64, __half>(p, st);
  return D == 128 ? launch<128, __nv_bfloat16>(p, st) : launch<64, __nv_bfloat16>(p, st);
}

}  // namespace pa
