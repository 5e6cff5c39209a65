// Attention of a ragged batch's rows to the keys of their entry (pa_fwd_cross)
// on the 5th-generation tensor cores (sm_103a): many rows a kv head, as whole
// target sequences have them.
//
// Mathematics as in cross.cu: softmax(scale Q K^T) V in one pass over the keys.
// The rows of a tile are packed over the G heads of a kv head (row i G + g of an
// entry; 128 / G whole tokens a tile), so that all rows of a CTA's two tiles share
// every K and V tile.  A row's reference m is the first 32 keys' largest score (so
// that a single key's P is exact) and follows larger ones, by whole numbers, only
// where they pass it by more than the slack of P's type: P and O are then scaled by
// powers of two, which is rare, and the exponentials do not wait for the maximum.
//
// Bound: the tensor cores, 4 D operations a (row, key) pair, and next to them the
// exponentials; with few rows the read of K and V.  Measured: 4 entries of 1024 rows
// and 4096 keys, 32 heads of 128: 202 to 206 us in a graph of a few launches (1.36 PFLOP/s, tensor
// pipe busy 58 %: a tile's chain of scores, softmax and values, two of them in turn), 217 to
// 225 us call by call, under the power cap (1.22 PFLOP/s); 64 of 8 rows and 4096
// masked keys, 32/8 heads of 128: 178 us (6.1 TB/s).  One persistent CTA an SM:
//   warps 0-7  softmax: one thread a row, group g = warp / 4 takes tile g
//   warp 8     K and Q tiles by TMA, warp 9 V tiles (one thread for both would hold K
//              back until V's place is free)
//   warp 10    issues O_g += P_g V (P_g from TMEM over S_g) and S_g = Q_g K^T
//   warp 11    limits of masked scores; clears rows of V that no row sees (0 times
//              what they hold may be NaN); tells that parts of cut streams are
//              written
// TMEM: S_0, S_1, O_0, O_1.  While one group's softmax runs, the tensor core works
// on the other group.  Where a pair has rows for one tile only, the groups take
// its tiles of keys in turn and their results are brought together at the end.
//
// Work: the streams (entry, kv head, pair of tiles) of up to 32 entries are dealt
// whole, the dearest first, to the CTAs in order and back again, where that comes
// within a join's time of equal shares.  Else they are laid end to end in 128-key
// tiles and dealt in equal shares, with cuts near an end of a stream moved there; a
// stream that is cut is joined by the CTA that finishes last.  The parts of a cut
// stream and its join are 8 to 15 thousand cycles of a CTA, as much as its tiles in
// a batch of a few hundred streams.  Whole and cut: 12 entries of 1 to 257 rows, 32/8
// heads of 128: 40.5 and 52 us; 32 of them: 84 and 103; 16 of 16 to 40 rows, 12 heads
// of 64: 21 and 26, the same with 2048 keys each: 35 and 31.
#include <type_traits>

#include "cross.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int kM = 128;  // rows of a query tile
constexpr int kN = 128;  // keys of a tile
constexpr int kSlab = 128 * 128;
constexpr int kSoft = 8;  // softmax warps
constexpr int kWarpK = 8, kWarpV = 9, kWarpMma = 10, kWarpFix = 11;
constexpr int kThreads = 12 * 32;
constexpr int kMinShare = 2;  // tiles
// Tiles that a cut moves to an end of its stream (0, 1, 2 and 4: 59, 57, 62 and 65 us
// for 12 entries of 1 to 257 rows), and what a stream's begin and end cost in tiles (0,
// 3 and 5: 69.5, 65 and 66 us; 32 entries of 24 rows 55, 40 and 41).
constexpr int kSnap = 1;
constexpr int kEnds = 3;
// Whole streams of a CTA at most (4 and 8: 103 and 84 us for 32 entries of 1 to 257
// rows), what a stream's begin and end cost (3 to 6 alike) and what a cut one's parts
// and join do (4: 54 us for what 8 to 24 do in 41; 16: 35 for what 8 does in 32), both
// in tiles of keys of one tile of rows.
constexpr int kRounds = 8;
constexpr int kWholeEnds = 4;
constexpr int kJoin = 8;

template <int D>
struct Layout {
  static constexpr int kTile = D / 64 * kSlab;
  static constexpr int kK = D == 128 ? 2 : 3;  // tiles of K
  static constexpr int kV = D == 128 ? 3 : 4;  // and of V, which stay longer
  static constexpr int kOffQ = 0;              // [2]
  static constexpr int kOffK = 2 * kTile;
  static constexpr int kOffV = kOffK + kK * kTile;
  static constexpr int kOffLimit = kOffV + kV * kTile;        // float [kV][kN] of scores
  static constexpr int kOffHalf = kOffLimit + kV * kN * 4;    // float2 [kM] m and l of a group
  static constexpr int kOffBar = kOffHalf + kM * 8;
  // q_full, q_empty; k_full, k_empty [kK]; v_full, v_ready, v_empty, l_full [kV]; s_full,
  // p_full, pv_done, o_free [2]; part_full [2], told
  static constexpr int kBars = 2 + 2 * kK + 4 * kV + 8 + 3;
  static constexpr int kOffSums = kOffBar + kBars * 8;        // int [kThreads / 32]
  static constexpr int kOffList = kOffSums + 12 * 4;          // int [kRounds][3] whole streams, -1
  static constexpr int kOffPlain = kOffList + kRounds * 12 + 4;   // int [kV] no limits in the tile
  static constexpr int kOffCut = kOffPlain + kV * 4;          // Cut [2]
  static constexpr int kOffMisc = kOffCut + 2 * 28;           // start [2], TMEM base
  static constexpr int kBytes = kOffMisc + 12;                // (the base is aligned to 1024)
  static_assert(kBytes <= 232448, "shared memory");
  static_assert(kOffLimit % 16 == 0 && kOffBar % 8 == 0, "read 16 bytes at a time; 64-bit words");
};

// P of the type: the largest score is brought to 2^shift at first, and may pass
// that by 2^slack before the reference moves.
template <typename T> struct Range;
template <> struct Range<__half> {  // up to 2^15, and 2^-32 of the largest still counts
  static constexpr float kShift = 8.f, kSlack = 7.f;
};
template <> struct Range<__nv_bfloat16> {
  static constexpr float kShift = 0.f, kSlack = 40.f;
};

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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float x;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(x) : "f"(a), "f"(b), "f"(c));
  return x;
}
// Ties the values of an asynchronous TMEM load to the wait in front of it.
__device__ __forceinline__ void arrived(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(v[i]));
}

// Scales the first `cols` columns of 16-bit probabilities in TMEM by 2^-k a lane,
// in two factors: one alone could lie below the type's range.
template <typename T>
__device__ __noinline__ void scale_p(uint32_t t, int cols, float by) {
  using E = Elem<T>;
  const float first = fmaxf(by, 0x1p-14f), second = fminf(by * 0x1p14f, 1.f);
  tc::tmem_wait_st();
#pragma unroll 1
  for (int c = 0; c < cols; c += 16) {
    float v[16];
    uint32_t w[16];
    tc::tmem_ld16(t + c, v);
    tc::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float2 x = E::to_f2(__float_as_uint(v[i]));
      x.x = x.x * first * second;
      x.y = x.y * first * second;
      w[i] = E::from_f2(x.x, x.y);
    }
    tc::tmem_st16u(t + c, w);
  }
  tc::tmem_wait_st();
}

__device__ __forceinline__ void mbar_arrive_2(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], 2;" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ float4 load16_l2(const void* src) {  // what another CTA has written
  float4 x;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "l"(src)
               : "memory");
  return x;
}

// Tokens of a tile, of a pair of tiles.
__device__ __forceinline__ int pair_tokens(const CrossParams& p) { return 2 * (kM / p.G); }
__device__ __forceinline__ int entry_pairs(const CrossParams& p, const CrossEntry& e) {
  const int n = pair_tokens(p);
  return (e.rows + n - 1) / n;
}
__device__ __forceinline__ int entry_tiles(const CrossEntry& e) {
  return max(1, (e.keys + kN - 1) / kN);  // (without keys: one, to write the empty rows)
}

// A part of a CTA's share: tiles [t0, t0 + n) of a stream.  A stream counts as its
// tiles and kEnds.  The cuts are at whole multiples of `share`; one that lies at most
// kSnap tiles behind a stream's begin counts as there, else one that lies at most kSnap
// in front of its end as there.  Of an entry's streams the pairs of one head lie as far
// apart as they can: side by side they would be one CTA's, one after the other, and
// each would read K and V from memory again (4 entries of 1024 rows and 4096 keys: 1.1
// GB of reads where K and V are 268 MB, 213 us; 202 this way).
struct Walk {
  int b, h, pair, t0, n, all, pairs;  // all: tiles of the stream; n = 0: no more
  int begin;                          // what the streams in front count
  int stop;                           // the cut behind the share; -1: none
  const int* list;                    // whole streams, or null
  CrossEntry e;

  __device__ __forceinline__ void open(const CrossParams& p, const int* at) {
    list = at;
    n = 0;
    if (*at < 0) return;
    b = at[0];
    h = at[1];
    pair = at[2];
    e = cross_entry(p, b, false);
    t0 = 0;
    n = all = entry_tiles(e);
  }

  __device__ __forceinline__ void take() {
    const int d = stop - begin;
    n = stop < 0 || d >= all ? all - t0 : d <= kSnap ? 0 : d >= all - kSnap ? all - t0 : d - t0;
  }
  __device__ __forceinline__ void next(const CrossParams& p) {
    if (list != nullptr) {
      open(p, list + 3);
      return;
    }
    if (t0 + n < all) {  // (cut)
      n = 0;
      return;
    }
    next_stream(p);
  }
  __device__ __forceinline__ void next_stream(const CrossParams& p) {
    n = 0;
    begin += all + kEnds;
    t0 = 0;
    if (++h == p.Hkv) {
      h = 0;
      if (++pair == pairs) {
        pair = 0;
        do {
          if (++b >= p.B) return;
          e = cross_entry(p, b, false);
          pairs = entry_pairs(p, e);
        } while (pairs == 0);
        all = entry_tiles(e);
      }
    }
    take();
  }
};

// Whether the streams are dealt whole, by one warp of every CTA in the same way: in
// descending order of their cost to CTAs 0, 1, .. and back again.  They are where the
// CTA with the most has no more than an equal share and a join.  (A lane has an entry
// and its pairs of tiles.  Divisions are left out where they can be: their code is
// cold.)
__device__ __noinline__ void deal_whole(const CrossParams& p, const CrossEntry e, const int pairs,
                                        const int tokens, int* scratch, int* list) {
  constexpr uint32_t kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31, ctas = (int)gridDim.x;
  const int tiles = entry_tiles(e);
  // the entry's pairs with rows for two tiles, and the last one if it has rows for one
  const int single = pairs > 0 && (2 * pairs - 1) * tokens >= e.rows ? 1 : 0;
  const int count0 = (pairs - single) * p.Hkv, count1 = single * p.Hkv;
  const int cost0 = count0 > 0 ? 2 * tiles + kWholeEnds : 0, cost1 = single ? tiles + kWholeEnds : 0;
  const int streams = __reduce_add_sync(kAll, count0 + count1);
  const unsigned all = __reduce_add_sync(kAll, (unsigned)count0 * cost0 + (unsigned)count1 * cost1);
  auto within = [&](int load) { return (long long)(load - kJoin) * ctas <= all; };
  if (lane <= kRounds) list[3 * lane] = -1;
  __syncwarp();
  // (no CTA has less than the dearest stream)
  if (streams == 0 || streams > kRounds * ctas ||
      !within(__reduce_max_sync(kAll, max(cost0, cost1)))) {
    if (lane == 0) list[1] = 0;
    return;
  }
  // kinds of streams in order; those of the lanes from `some` on, without an entry,
  // have no streams and are last
  const int some = (p.B + 7) / 8 * 8, over = max(0, lane - some);
  int rank0 = over, rank1 = over + (cost1 == 0 ? 32 - some : 0);
#pragma unroll 1
  for (int k0 = 0; k0 < some; k0 += 8)
#pragma unroll
    for (int k = k0; k < k0 + 8; ++k) {
      const int a = __shfl_sync(kAll, cost0, k), b = __shfl_sync(kAll, cost1, k);
      rank0 += (a > cost0 || (a == cost0 && k < lane)) + (b > cost0);
      rank1 += (a >= cost1) + (b > cost1 || (b == cost1 && k < lane));
    }
  // {entry, cost, pairs a head, first pair}; streams of the kind, then those in front
  int4* kind = reinterpret_cast<int4*>(scratch);  // [64]
  int* count = scratch + 4 * 64;                  // [64]
  kind[rank0] = make_int4(lane, cost0, pairs - single, 0);
  count[rank0] = count0;
  kind[rank1] = make_int4(lane, cost1, 1, pairs - 1);
  count[rank1] = count1;
  __syncwarp();
  const int2 c = reinterpret_cast<int2*>(count)[lane];
  int upto = c.x + c.y;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kAll, upto, o);
    if (lane >= o) upto += x;
  }
  reinterpret_cast<int2*>(count)[lane] = make_int2(upto - c.x - c.y, upto - c.y);
  __syncwarp();
  // the loads of 31 CTAs spread over the order and, in the last lane, the CTA's own
  const int cta = lane == 31 ? (int)blockIdx.x : lane * (ctas - 1) / 30;
  int load = 0;
#pragma unroll 1
  for (int r = 0; r < kRounds; ++r) {
    const int i = r * ctas + (r & 1 ? ctas - 1 - cta : cta);
    if (i >= streams) break;
    int k = 0;  // (kinds without streams are behind the last)
#pragma unroll
    for (int step = 32; step > 0; step >>= 1)
      if (count[k + step] <= i) k += step;
    const int4 x = kind[k];
    load += x.y;
    if (lane == 31) {
      const int off = i - count[k];
      const int h = (int)__fdividef((float)off + 0.5f, (float)x.z);  // (exact: off < 2^20)
      list[3 * r] = x.x;
      list[3 * r + 1] = h;
      list[3 * r + 2] = x.w + off - h * x.z;
    }
  }
  // (of the same CTAs in all of them: every CTA comes to the same answer)
  const bool whole = within(__reduce_max_sync(kAll, lane < 31 ? load : 0));
  if (lane == 31) {
    if (!whole) list[0] = -1;
    if (list[0] < 0) list[1] = whole ? 1 : 0;
  }
  fence_proxy_async_smem();  // (the scratch is V's place)
}

// What a join needs of a cut stream: its rows and the CTAs of its parts.
struct Cut {
  int q0, rows, h, pair, cta0, cta1, last;
};
static_assert(sizeof(Cut) == 28, "kOffCut");

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    wide_kernel(const __grid_constant__ CrossParams p, const __grid_constant__ CUtensorMap tmq,
                const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  using L = Layout<D>;
  using E = Elem<T>;
  using R = Range<T>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  if ((smem_u32(smem) & 1023) != 0) {  // (what swizzled tiles ask for; no room is left to move them)
    if (threadIdx.x == 0) report(p.err, PA_DEVERR_TIMEOUT, -1, 99);
    return;
  }
  uint8_t* sQ = smem + L::kOffQ;
  uint8_t* sK = smem + L::kOffK;
  uint8_t* sV = smem + L::kOffV;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 1;
  uint64_t* k_full = bars + 2;
  uint64_t* k_empty = k_full + L::kK;
  uint64_t* v_full = k_empty + L::kK;
  uint64_t* v_ready = v_full + L::kV;
  uint64_t* v_empty = v_ready + L::kV;
  uint64_t* l_full = v_empty + L::kV;  // the tile's limits
  uint64_t* s_full = l_full + L::kV;
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 2;
  uint64_t* o_free = pv_done + 2;
  uint64_t* part_full = o_free + 2;           // [2]: the rows of the first, last part are written
  uint64_t* told = part_full + 2;             // what is to be joined is known
  int* sSums = reinterpret_cast<int*>(smem + L::kOffSums);
  Cut* sCut = reinterpret_cast<Cut*>(smem + L::kOffCut);       // the first part, the last
  int* sStart = reinterpret_cast<int*>(smem + L::kOffMisc);    // entry, tiles in front of it
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc + 8);
  float* sLimit = reinterpret_cast<float*>(smem + L::kOffLimit);
  float2* sHalf = reinterpret_cast<float2*>(smem + L::kOffHalf);
  int* sPlain = reinterpret_cast<int*>(smem + L::kOffPlain);
  int* sList = reinterpret_cast<int*>(smem + L::kOffList);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < L::kK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < L::kV; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_ready[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&l_full[i], 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&s_full[g], 1);
      mbar_init(&p_full[g], kSoft / 2);
      mbar_init(&pv_done[g], 1);
      mbar_init(&o_free[g], kSoft);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&part_full[i], kSoft);
    mbar_init(told, 1);
    fence_mbar_init();
  }

  if (tid == 32) {
    tma_prefetch_desc(&tmq);
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  // TMEM is taken behind the wait (a kernel in front may have yet to take its own),
  // and a dependent grid may start once it is taken.
  griddep_wait();
  if (warp == kWarpMma) {
    tc::tmem_alloc(tslot, 512);
    tc::tmem_relinquish();
  }
  // ---- the CTA's share: the tiles of all entries, then the entry it begins in.  Up
  // to 32 entries every warp finds them by itself.
  int total = 0, share = 0, start = 0, b_start = 0, b_begin = 0;
  {
    CrossEntry e = {};
    int pairs = 0;
    auto cost_of = [&](int b, bool rep) {
      if (b >= p.B) return 0;
      e = cross_entry(p, b, rep);
      pairs = entry_pairs(p, e);
      return pairs * p.Hkv * (entry_tiles(e) + kEnds);
    };
    auto upto = [&](int x) {  // with the lanes in front
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      return x;
    };
    auto deal = [&]() {
      share = max(kMinShare, (total + (int)gridDim.x - 1) / (int)gridDim.x);
      start = share * (int)blockIdx.x;
    };
    if (p.B <= 32) {
      const int cost = cost_of(lane, warp == 0 && blockIdx.x == 0);
      if (warp == kWarpFix) deal_whole(p, e, pairs, kM / p.G, reinterpret_cast<int*>(sV), sList);
      const int x = upto(cost);
      total = __shfl_sync(0xffffffffu, x, 31);
      deal();
      const uint32_t mine = __ballot_sync(0xffffffffu, start >= x - cost && start < x);
      b_start = mine != 0 ? __ffs((int)mine) - 1 : 0;
      b_begin = __shfl_sync(0xffffffffu, x - cost, b_start);
    } else {
      if (tid < 2) sList[tid] = tid - 1;
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        int before = 0;
#pragma unroll 1
        for (int b0 = 0; b0 < p.B; b0 += kThreads) {
          const int cost = cost_of(b0 + tid, pass == 0 && blockIdx.x == 0);
          int x = upto(cost);
          __syncthreads();  // (sSums have been read)
          if (lane == 31) sSums[warp] = x;
          __syncthreads();
          const int sum = lane < kThreads / 32 ? sSums[lane] : 0;
          x += before + __reduce_add_sync(0xffffffffu, lane < warp ? sum : 0);
          before += __reduce_add_sync(0xffffffffu, sum);
          if (pass == 1 && start >= x - cost && start < x) {
            sStart[0] = b0 + tid;
            sStart[1] = x - cost;
          }
        }
        if (pass == 0) {
          total = before;
          deal();
        }
      }
      __syncthreads();
      b_start = start < total ? sStart[0] : 0;
      b_begin = start < total ? sStart[1] : 0;
    }
  }
  Walk at;
  at.n = 0;
  at.list = nullptr;
  if (start < total) {
    at.b = b_start;
    at.e = cross_entry(p, at.b, false);
    at.pairs = entry_pairs(p, at.e);
    at.all = entry_tiles(at.e);
    at.stop = start + share < total ? start + share : -1;
    const int off = start - b_begin, stream = off / (at.all + kEnds);
    at.begin = b_begin + stream * (at.all + kEnds);
    at.t0 = off - stream * (at.all + kEnds);
    at.pair = stream / p.Hkv;
    at.h = stream - at.pair * p.Hkv;
    if (at.t0 < at.all && at.t0 <= kSnap) at.t0 = 0;
    if (at.t0 > 0 && at.t0 >= at.all - kSnap) at.next_stream(p);
    else at.take();
  }
  const int tokens = kM / p.G, tile_rows = tokens * p.G;

  // rows of a Q tile that no token fills stay zero
  if (tile_rows < kM) {
    for (int i = tid; i < 2 * L::kTile / 16; i += kThreads)
      *reinterpret_cast<uint4*>(sQ + i * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  griddep_launch_dependents();
  if (sList[0] >= 0 || sList[1] != 0) at.open(p, sList);
  const uint32_t tbase = *tslot;
  if (tid < 2) sCut[tid].last = 0;  // (before the first part's end, which is behind barriers)
  auto tS = [&](int g) { return tbase + (uint32_t)(g * 128); };
  auto tO = [&](int g) { return tbase + 256u + (uint32_t)(g * D); };
  // One tile of rows: the groups take its tiles of keys in turn.
  auto solo = [&](const Walk& w) { return (2 * w.pair + 1) * tokens >= w.e.rows; };

  bool failed = false;
  auto wait = [&](uint64_t* bar, uint32_t par, int where) {
    if (!failed && !mbar_wait(bar, par)) {
      report(p.err, PA_DEVERR_TIMEOUT, -1, where);
      failed = true;
    }
  };

  if (warp == kWarpK || warp == kWarpV) {
    // ======================= K and Q, V =======================
    const bool is_v = warp == kWarpV;
    const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
    uint64_t* full = is_v ? v_full : k_full;
    uint64_t* empty = is_v ? v_empty : k_empty;
    uint8_t* ring = is_v ? sV : sK;
    const CUtensorMap* map = is_v ? &tmv : &tmk;
    const int stages = is_v ? L::kV : L::kK;
    int s = 0, a = 0;     // place in the ring,
    uint32_t round = 0;   // and how often it has come round
    int behind = 0;       // tiles issued, up to the ring's places
    if (lane == 0) {
      for (; at.n > 0; at.next(p)) {
        if (at.e.keys == 0) continue;
        for (int t = at.t0; t < at.t0 + at.n; ++t) {
          wait(&empty[s], (round & 1) ^ 1, is_v ? 21 : 20);
          if (failed) break;
          mbar_arrive_expect_tx(&full[s], L::kTile);
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(ring + s * L::kTile + c * kSlab, map, &full[s], c * 64, at.h / p.kv_split,
                        at.e.k0 + t * kN, 0, keep);
          if (++s == stages) {
            s = 0;
            ++round;
          }
          behind = min(behind + 1, stages);
          if (!is_v && t == at.t0) {
            if (a >= 1) wait(q_empty, (uint32_t)((a - 1) & 1), 10);
            if (failed) break;
            const int q_tiles = solo(at) ? 1 : 2;
            mbar_arrive_expect_tx(q_full, (uint32_t)(q_tiles * (D / 64) * tile_rows * 128));
            for (int g = 0; g < q_tiles; ++g)
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(sQ + g * L::kTile + c * kSlab, &tmq, q_full, c * 64, at.h * p.G,
                            at.e.q0 + (2 * at.pair + g) * tokens, 0, once);
          }
        }
        ++a;
      }
      // every copy must land before the CTA leaves: the last `behind` tiles
      for (int i = 0; i < behind; ++i) {
        if (s-- == 0) {
          s = stages - 1;
          --round;
        }
        if (failed) mbar_wait(&full[s], round & 1);
        else wait(&empty[s], round & 1, 30);
      }
    }
    __syncwarp();
  } else if (warp == kWarpFix) {
    // ======================= limits of scores, rows of V that no row sees =====
    int k = 0, parts = 0;
    // The softmax warps do not wait until their part's writes have arrived: this warp
    // arrives for the CTA some time later.
    Cut cut = {};
    int pending = -1;  // the part: 0 first, 1 last
    auto tell = [&]() {
      if (pending < 0) return;
      wait(&part_full[pending], 0, 27);
      if (lane == 0) {
        __threadfence();
        cut.last = arrive_last(p.words + cut.cta0, launch_tag(), cut.cta1 - cut.cta0 + 1) ? 1 : 0;
        __threadfence();
        sCut[pending] = cut;
      }
      __syncwarp();
      pending = -1;
    };
    for (; at.n > 0; at.next(p)) {
      if (at.e.keys == 0) continue;
      // The mask of the lane's four keys of a tile is read two tiles ahead and looked at
      // only then: while the memory is busy with K and V a byte takes as long as a tile.
      uint32_t mask[2][kN / 32];
      auto read_mask = [&](int t, uint32_t (&x)[kN / 32]) {
#pragma unroll
        for (int c = 0; c < kN / 32; ++c) {
          const int key = t * kN + c * 32 + lane;
          x[c] = 1;
          if (p.key_mask != nullptr && key < at.e.keys) x[c] = load_byte(p.key_mask + at.e.k0 + key);
        }
      };
      read_mask(at.t0, mask[0]);
      read_mask(at.t0 + 1, mask[1]);
#pragma unroll 1
      for (int t = at.t0; t < at.t0 + at.n; ++t, ++k) {
        const int s = k % L::kV;
        uint32_t seen = 0;
#pragma unroll
        for (int c = 0; c < kN / 32; ++c) {
          if (t * kN + c * 32 + lane < at.e.keys && mask[0][c] != 0) seen |= 1u << c;
          mask[0][c] = mask[1][c];
        }
        const bool whole = __all_sync(0xffffffffu, seen == 0xfu);
        // V's place is free, so the limits of the last tile in it are used up; the
        // softmax warps can go on while V is on its way
        wait(&v_empty[s], (uint32_t)((k / L::kV & 1) ^ 1), 24);
        if (lane == 0) sPlain[s] = whole ? 1 : 0;
        if (!whole) {
#pragma unroll
          for (int c = 0; c < kN / 32; ++c)
            sLimit[s * kN + c * 32 + lane] = seen >> c & 1 ? -neg_inf() : neg_inf();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&l_full[s]);
        if (t + 2 < at.t0 + at.n) read_mask(t + 2, mask[1]);
        wait(&v_full[s], (uint32_t)(k / L::kV & 1), 25);
        if (!whole) {
          uint8_t* tile = sV + s * L::kTile;
          // the lane's four rows, each lane's chunks in another order
#pragma unroll 4
          for (int i = 0; i < D / 8; ++i) {
            uint8_t* to = tile + (i >> 3) * kSlab + lane * 128 + (((i ^ lane) & 7) << 4);
#pragma unroll
            for (int c = 0; c < kN / 32; ++c)
              if ((seen >> c & 1) == 0)
                *reinterpret_cast<uint4*>(to + c * 32 * 128) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_ready[s]);
        if (pending >= 0 && __all_sync(0xffffffffu, mbar_try_wait(&part_full[pending], 0))) tell();
      }
      if (at.t0 > 0 || at.n < at.all) {
        tell();
        pending = at.t0 == 0 ? 1 : 0;
        cut = {at.e.q0, at.e.rows, at.h, at.pair, (at.begin + min(kSnap, at.all - 1)) / share, 0, 0};
        cut.cta1 = max(cut.cta0, (at.begin + at.all - kSnap - 1) / share);
        ++parts;
      }
    }
    tell();
    if (parts > 0 && lane == 0) mbar_arrive(told);
  } else if (warp == kWarpMma) {
    // ======================= MMA issuer =======================
    // Per tile and group: O_g += P_g V, then S_g of the next tile.  One thread's
    // MMAs run in the order it issues them, so S_g may follow the product that
    // reads P_g from the same columns without a wait.  The warp issues as one, an
    // elected thread's predicate on, with operands broadcast to uniform registers.
    constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
    const uint32_t id_s = tc::idesc_f16(kM, kN, bf, false);
    const uint32_t id_o = tc::idesc_f16(kM, D, bf, true);
    const uint64_t d16 = tc::smem_desc(0, 16, 1024), dslab = tc::smem_desc(0, kSlab, 1024);
    const uint32_t qlo = (uint32_t)d16 + (smem_u32(sQ) >> 4), klo = (uint32_t)d16 + (smem_u32(sK) >> 4);
    const uint32_t vlo = (uint32_t)dslab + (smem_u32(sV) >> 4);
    auto desc = [](uint64_t base, uint32_t lo) {
      uint64_t d;
      asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"((uint32_t)(base >> 32)));
      return d;
    };
    auto uni = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
    uint32_t on;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(on));
    const uint32_t tb = uni(tbase);
    int k = 0, a = 0, n0 = 0, n1 = 0, m0 = 0, m1 = 0;
    auto scores = [&](int g, int q_tile, int s) {
      const uint32_t q0 = uni(qlo + (uint32_t)((q_tile * L::kTile) >> 4));
      const uint32_t k0 = uni(klo + (uint32_t)((s * L::kTile) >> 4));
      const uint32_t ts = uni(tb + g * 128);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * kSlab + (kk & 3) * 32) >> 4;
        mma_ss_if(on, ts, desc(d16, q0 + off), desc(d16, k0 + off), id_s, kk > 0);
      }
      commit_if(on, &s_full[g]);
      __syncwarp();
    };
    auto release = [&](uint64_t* bar) {
      commit_if(on, bar);
      __syncwarp();
    };
    auto values = [&](int g, int s, bool add) {  // O_g (+)= P_g V
      const uint32_t v0 = uni(vlo + (uint32_t)((s * L::kTile) >> 4));
      const uint32_t ts = uni(tb + g * 128), to = uni(tb + 256 + g * D);
      const uint32_t more = uni(add);
#pragma unroll
      for (int kk = 0; kk < kN / 16; ++kk)
        mma_ts_if(on, to, ts + kk * 8, desc(dslab, v0 + (kk * 2048 >> 4)), id_o, kk > 0 ? 1u : more);
      commit_if(on, &pv_done[g]);
      __syncwarp();
    };
    for (; at.n > 0; at.next(p)) {
      if (at.e.keys == 0) continue;
      // steps of the part: (tile, group), a tile's two groups or one of them
      const bool one = solo(at);
      wait(q_full, (uint32_t)(a & 1), 40);
      auto first = [&](int g, int t, bool last_of_tile) {
        const int s = (k + t) % L::kK;
        wait(&k_full[s], (uint32_t)((k + t) / L::kK & 1), 41);
        tc::fence_after_sync();
        scores(g, one ? 0 : g, s);
        if (last_of_tile) release(&k_empty[s]);
        if (last_of_tile && t == at.n - 1) release(q_empty);  // the part's last scores
      };
      first(0, 0, one);
      if (!one) first(1, 0, true);
      else if (at.n > 1) first(1, 1, true);
#pragma unroll 1
      for (int i = 0; i < (one ? at.n : 2 * at.n); ++i) {
        const int g = i & 1, t = one ? i : i >> 1, next_t = one ? i + 2 : t + 1;
        const int s = (k + t) % L::kV;
        const int n = g ? n1 : n0, m = g ? m1 : m0;
        const bool fresh = one ? i < 2 : t == 0;
        if (one || g == 0) wait(&v_ready[s], (uint32_t)((k + t) / L::kV & 1), 50);
        wait(&p_full[g], (uint32_t)(n & 1), 51 + g);
        if (fresh && m >= 1) wait(&o_free[g], (uint32_t)((m - 1) & 1), 53 + g);
        tc::fence_after_sync();
        values(g, s, !fresh);
        if (g) ++n1;
        else ++n0;
        if (next_t < at.n) first(g, next_t, one || g == 1);
        if (one || g == 1) release(&v_empty[s]);
      }
      k += at.n;
      ++a;
      ++m0;
      ++m1;
    }
  } else {
    // ======================= softmax =======================
    const int g = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const float f = p.scale_log2;
    // 32 columns of a row a thread: four threads exchange 16-byte chunks, so that each
    // has the same chunk of their four rows, and 64 bytes of a row are written at a time
    auto write = [&](long long my_row, int col, const float (&x)[32], float by) {
      uint4 c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[i] = make_uint4(E::from_f2(x[8 * i] * by, x[8 * i + 1] * by),
                          E::from_f2(x[8 * i + 2] * by, x[8 * i + 3] * by),
                          E::from_f2(x[8 * i + 4] * by, x[8 * i + 5] * by),
                          E::from_f2(x[8 * i + 6] * by, x[8 * i + 7] * by));
#pragma unroll
      for (int bit = 1; bit < 4; bit *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i & bit) continue;
          const bool up = (lane & bit) != 0;
          uint4 send = up ? c[i] : c[i | bit];
          send.x = __shfl_xor_sync(0xffffffffu, send.x, bit);
          send.y = __shfl_xor_sync(0xffffffffu, send.y, bit);
          send.z = __shfl_xor_sync(0xffffffffu, send.z, bit);
          send.w = __shfl_xor_sync(0xffffffffu, send.w, bit);
          if (up) c[i] = send;
          else c[i | bit] = send;
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long to = __shfl_sync(0xffffffffu, my_row, (lane & 28) + i);
        if (to >= 0)
          *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.out) + to * D + col + (lane & 3) * 8) = c[i];
      }
    };
    auto weight = [](float2 x, float ref) {
      return x.y == 0.f ? 0.f : x.x == ref ? 1.f : ex2(x.x - ref);
    };
    int done[2] = {0, 0}, k = 0;  // tiles of either group, of the CTA
    bool cut = false;
    for (; at.n > 0; at.next(p)) {
      const bool one = solo(at);
      const int tile = one ? 0 : g;  // the group's rows
      const int token = (2 * at.pair + tile) * tokens + r / p.G, head = at.h * p.G + r % p.G;
      const bool valid = r < tile_rows && token < at.e.rows;
      float m = neg_inf(), l = 0.f;
      int n = g ? done[1] : done[0];
      for (int j = one ? g : 0; j < at.n && at.e.keys > 0; j += one ? 2 : 1) {
        bool whole = p.key_mask == nullptr && (at.t0 + j + 1) * kN <= at.e.keys;
        const int place = (k + j) % L::kV;
        wait(&s_full[g], (uint32_t)(n & 1), 60 + g);
        // (behind the scores: P V of the last tile in this place has been issued then)
        if (!whole) {
          wait(&l_full[place], (uint32_t)((k + j) / L::kV & 1), 66);
          whole = sPlain[place] != 0;
        }
        tc::fence_after_sync();
        const uint32_t ts = tS(g) + lane_off;
        uint64_t sum2[4] = {0, 0, 0, 0};  // four pairs of sums
        float alpha = 1.f;
        float v[32];
        // 32 scores at a time, in a rolled loop (unrolled, the roles' code passes
        // what the instruction caches hold)
        auto probabilities = [&](auto masked, int key0) {
          if constexpr (masked) {
            // -inf where a key is not seen, whatever the score is (NaN too), else at most inf
            const float4* limit = reinterpret_cast<const float4*>(sLimit + place * kN + key0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 x = limit[i];
              v[4 * i] = fminf(v[4 * i], x.x);
              v[4 * i + 1] = fminf(v[4 * i + 1], x.y);
              v[4 * i + 2] = fminf(v[4 * i + 2], x.z);
              v[4 * i + 3] = fminf(v[4 * i + 3], x.w);
            }
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
              const float e0 = ex2(z.x), e1 = ex2(z.y);
              more[e & 3] = e < 4 ? pair(e0, e1) : add2(more[e & 3], pair(e0, e1));
              top4[e & 3] = e < 4 ? fmaxf(v[2 * e], v[2 * e + 1])
                                  : max3(top4[e & 3], v[2 * e], v[2 * e + 1]);
              pk[e] = E::from_f2(e0, e1);
            }
            const float top = max3(fmaxf(top4[0], top4[1]), top4[2], top4[3]) * f;
            const bool far = top > m + (R::kShift + R::kSlack);
            if (!__any_sync(0xffffffffu, far)) break;
            float by = 1.f;
            if (far) {
              if (m == neg_inf()) {
                m = top - R::kShift;
              } else {
                const float up = ceilf(top - m) - R::kShift;
                by = ex2(-up);
                m += up;
              }
            }
            alpha *= by;
            l *= by;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 z = halves(sum2[i]);
              sum2[i] = pair(z.x * by, z.y * by);
            }
            scale_p<T>(ts, key0 / 2, by);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) sum2[i] = add2(sum2[i], more[i]);
          tc::tmem_st16u(ts + key0 / 2, pk);  // over scores that have been used
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
        if (whole) row(std::false_type{});
        else row(std::true_type{});
        const float2 sum = halves(add2(add2(sum2[0], sum2[1]), add2(sum2[2], sum2[3])));
        l += sum.x + sum.y;
        if (j >= (one ? 2 : 1) && __any_sync(0xffffffffu, alpha != 1.f)) {
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
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[g]);
        ++n;
      }

      if (at.e.keys > 0) {
        k += at.n;
        done[0] += one ? (at.n + 1) / 2 : at.n;
        done[1] += one ? at.n / 2 : at.n;
      }

      // ---- the part's result: the group's rows, or half of the columns of the one
      // tile's rows, whose results are those of both groups
      const bool whole = at.t0 == 0 && at.n == at.all;
      const int col0 = one ? g * (D / 2) : 0, cols = one ? D / 2 : D;
      const long long my_row = valid ? (long long)(at.e.q0 + token) * p.Hq + head : -1;
      auto put_lse = [&](float ref, float sum) {
        if (valid && (!one || g == 0) && p.lse != nullptr)
          p.lse[(int64_t)head * p.total_q + at.e.q0 + token] =
              sum == 0.f ? neg_inf() : (ref + log2f(sum)) * kLn2;
      };
      if (at.e.keys == 0) {
        float zero[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) zero[e] = 0.f;
#pragma unroll 1
        for (int col = col0; col < col0 + cols; col += 32) write(my_row, col, zero, 0.f);
        put_lse(m, l);
        continue;
      }
      // What O_0 and O_1 count for (a part without a seen key counts for nothing,
      // and its O may hold nothing).
      float2 half[2] = {make_float2(m, l), make_float2(m, l)};
      if (one) {
        // (each group's in turn, in one place)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (g == x) sHalf[r] = half[g];
          named_barrier(1, 256);
          if (g != x) half[x] = sHalf[r];
          if (x == 0) named_barrier(1, 256);
        }
        m = fmaxf(half[0].x, half[1].x);
      }
      const float weight0 = weight(half[0], m), weight1 = weight(half[1], m);
      if (one) l = fmaf(weight0, half[0].y, weight1 * half[1].y);
      // P V of either group's last tile (the other group's softmax of it is done)
      if (one || g == 0) wait(&pv_done[0], (uint32_t)((done[0] - 1) & 1), 64);
      if (one ? at.n > 1 : g == 1) wait(&pv_done[1], (uint32_t)((done[1] - 1) & 1), 65);
      tc::fence_after_sync();
      const float by = l == 0.f ? 0.f : 1.f / l;
      const int slot = 2 * blockIdx.x + (at.t0 == 0 ? 1 : 0);
      const int64_t my_part = ((int64_t)slot * 2 + tile) * kM;
#pragma unroll 1
      for (int col = col0; col < col0 + cols; col += 32) {
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0.f;
#pragma unroll 1
        for (int x = one ? 0 : g; x < (one ? min(at.n, 2) : g + 1); ++x) {
          float y[32];
          tc::tmem_ld32(tO(x) + lane_off + col, y);
          tc::tmem_wait_ld();
          arrived(y);
          const float w = x ? weight1 : weight0;
          if ((x ? half[1] : half[0]).y != 0.f) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = fmaf(w, y[e], o[e]);
          }
        }
        if (whole) {
          write(my_row, col, o, by);
        } else if (valid) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(p.part_o + (my_part * (D / 4) + (col / 4 + e) * kM + r) * 4) =
                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (one) {
          mbar_arrive(&o_free[0]);
          mbar_arrive(&o_free[1]);
        } else {
          mbar_arrive_2(&o_free[g]);
        }
      }
      if (whole) {
        put_lse(m, l);
        continue;
      }
      if (valid && (!one || g == 0)) p.part_ml[my_part + r] = make_float2(m, l);
      cut = true;
      __syncwarp();
      if (lane == 0) mbar_arrive(&part_full[at.t0 == 0 ? 1 : 0]);
    }

    // ---- joins: of streams whose last part was this CTA's
    if (cut) {
      wait(told, 0, 68);
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        const Cut c = sCut[x];
        if (!c.last) continue;
        const bool one = (2 * c.pair + 1) * tokens >= c.rows;
        const int tile = one ? 0 : g;
        const int token = (2 * c.pair + tile) * tokens + r / p.G, head = c.h * p.G + r % p.G;
        const bool valid = r < tile_rows && token < c.rows;
        const int col0 = one ? g * (D / 2) : 0, cols = one ? D / 2 : D;
        const long long my_row = valid ? (long long)(c.q0 + token) * p.Hq + head : -1;
        // the row tile's place in part `cta`
        auto from = [&](int cta) {
          return ((int64_t)(2 * cta + (cta == c.cta0 ? 1 : 0)) * 2 + tile) * kM;
        };
        // 64 columns at a time (32 where there are no more): what a part has of them is
        // one wait for L2
        constexpr int kAtOnce = D == 128 ? 16 : 8;
#pragma unroll 1
        for (int col = col0; col < col0 + cols; col += 4 * kAtOnce) {
          float ref = neg_inf(), sum = 0.f;
          float4 acc[kAtOnce];
#pragma unroll
          for (int e = 0; e < kAtOnce; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (valid) {
#pragma unroll 1
            for (int cta = c.cta0; cta <= c.cta1; ++cta) {
              float4 y[kAtOnce];
              const float2 ml = __ldcg(p.part_ml + from(cta) + r);
#pragma unroll
              for (int e = 0; e < kAtOnce; ++e)
                y[e] = load16_l2(p.part_o + (from(cta) * (D / 4) + (col / 4 + e) * kM + r) * 4);
              // (a part without a seen key counts for nothing, its O may hold nothing)
              if (ml.y == 0.f) continue;
              const float to = fmaxf(ref, ml.x);
              const float v = ref == to ? 1.f : ex2(ref - to), w = ml.x == to ? 1.f : ex2(ml.x - to);
              ref = to;
              sum = fmaf(sum, v, w * ml.y);
#pragma unroll
              for (int e = 0; e < kAtOnce; ++e) {
                acc[e].x = fmaf(acc[e].x, v, w * y[e].x);
                acc[e].y = fmaf(acc[e].y, v, w * y[e].y);
                acc[e].z = fmaf(acc[e].z, v, w * y[e].z);
                acc[e].w = fmaf(acc[e].w, v, w * y[e].w);
              }
            }
          }
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          if (valid && col == 0 && p.lse != nullptr)
            p.lse[(int64_t)head * p.total_q + c.q0 + token] =
                sum == 0.f ? neg_inf() : (ref + log2f(sum)) * kLn2;
          __syncwarp();
#pragma unroll
          for (int x = 0; x < kAtOnce; x += 8) {
            float o[32];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              o[4 * e] = acc[x + e].x;
              o[4 * e + 1] = acc[x + e].y;
              o[4 * e + 2] = acc[x + e].z;
              o[4 * e + 3] = acc[x + e].w;
            }
            write(my_row, col + 4 * x, o, inv);
          }
        }
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kWarpMma) tc::tmem_dealloc(tbase, 512);
}

template <int D, typename T>
cudaError_t launch(const CrossParams& p, const CUtensorMap& tmq, const CUtensorMap& tmk,
                   const CUtensorMap& tmv, cudaStream_t st) {
  static std::atomic<uint64_t> devices{0};
  const cudaError_t e = allow_shared(reinterpret_cast<const void*>(wide_kernel<D, T>),
                                     Layout<D>::kBytes, &devices);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)num_sms());
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Layout<D>::kBytes;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  overlap_launch(&at);
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, wide_kernel<D, T>, p, tmq, tmk, tmv);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

// Of each CTA: an arrival word; m, l and O of two parts of two tiles.
size_t cross_wide_workspace(int D) {
  const size_t rows = (size_t)num_sms() * 2 * 2 * kM;
  return align256((size_t)num_sms() * 8) + align256(rows * 8) + rows * D * 4;
}

cudaError_t launch_cross_wide(CrossParams p, const CUtensorMap& tmq, const CUtensorMap& tmk,
                              const CUtensorMap& tmv, int D, int dtype, void* workspace,
                              cudaStream_t st) {
  const size_t rows = (size_t)num_sms() * 2 * 2 * kM;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.words = reinterpret_cast<unsigned long long*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + align256((size_t)num_sms() * 8));
  p.part_o = reinterpret_cast<float*>(ws + align256((size_t)num_sms() * 8) + align256(rows * 8));
  if (D == 64)
    return dtype == PA_F16 ? launch<64, __half>(p, tmq, tmk, tmv, st)
                           : launch<64, __nv_bfloat16>(p, tmq, tmk, tmv, st);
  return dtype == PA_F16 ? launch<128, __half>(p, tmq, tmk, tmv, st)
                         : launch<128, __nv_bfloat16>(p, tmq, tmk, tmv, st);
}

}  // namespace pa
