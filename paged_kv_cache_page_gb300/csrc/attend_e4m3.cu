// Attention of a ragged batch over a paged e4m3 cache (sm_103a): single
// tokens and short query blocks, split over the keys.  The interface is that
// of the mixed launch of vLLM #6052 "Unify the kernel used in flash attention
// backend"; the cache holds 8-bit values with a scale for each kv head.
//
// Mathematics.  For a query row q (head h of kv head j) over its visible keys
//   s_t = (scale ks_j) q . K_t,  O = vs_j sum_t e^{s_t - LSE} V_t,
// computed as one pass with a running reference m (log2 domain) and sum l.
// e4m3 values are exact in fp16, so both products run on fp16 tensor-core
// MMAs with fp32 accumulation.  fp16 q is used as it is; a bf16 q row is
// first scaled by a power of two to a largest magnitude in [1, 2), which
// leaves every bf16 significand exact and loses only what lies 2^-24 below
// the row's largest value.  Probabilities are rounded to fp16 (half a unit is
// 2^-12) as 2^(s - m + 10): the ten powers of two move the smallest normal
// fp16 probability from 2^-14 to 2^-24 of the row's largest.  m follows the
// maximum only when it is passed by 2^5, so that p stays below 2^15 and the
// accumulators are hardly ever rescaled; l sums the unrounded values in fp32.
//
// Bound: HBM, 2 D bytes a key and kv head; half of a 16-bit cache's.  256
// streams of 4096 keys of 32 kv heads, D = 128, run in 1.28 ms, 6.7 TB/s; 64
// streams of 4096 keys of 8 kv heads in 102 us, 5.3 TB/s; shorter calls are
// bound by latency (8 streams of 1024 to 8192 keys: 24.9 us, 3.0 TB/s; 1 of
// 4096: 15 us; 2 of 100: 6.3 us): launch, lengths, table, keys, join, and the way
// of code that runs once.  A warp takes units of 16 keys, two at a time where
// it has two -- twice the independent work for the same waits:
//   copy     cp.async 16 bytes a lane into the warp's own ring of stages --
//            no producer warp, no barrier: a warp waits for its own copies
//   S        [16 rows][16 keys] = Q K^T, MMAs m16n8k16, Q in registers.  A
//            lane's 16 bytes of a key are four MMAs' operands as they stand:
//            which feature an MMA calls k is free, as long as Q agrees
//   softmax  in the accumulator fragments, which are PV's operand layout
//   O        [16 rows][D] += P V: V's operand pairs two keys' bytes (a byte
//            permute), then the same conversion
// The 16-byte slots of a stage are permuted so that both reads touch every
// bank once.
//
// Work.  The streams (sequence, kv head, 16-row tile) are laid end to end in
// units of 16 keys and dealt to the CTAs -- whole, in slots or in equal shares,
// below; the cut is made on the GPU from the lengths.  A CTA has at most one
// stream that began earlier and one that goes on, so two partial results a CTA
// hold every split, and the CTA that finishes a split stream last merges it.
// The 128 bytes of a key of one kv head lie Hkv D apart, too short a run for
// DRAM: a CTA therefore takes up to eight neighbouring kv heads side by side.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attend_e4m3.cuh"

namespace pa {
int set_error(int code, const char* fmt, ...);

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;       // query rows of a tile
constexpr int kKeys = 16;       // keys of a unit
constexpr int kMaxB = 4096;
constexpr float kShift = kE4m3Shift, kSlack = kE4m3Slack;
// The limits of the dealing, with both sides on 8 kv heads of D = 128 unless said
// otherwise (us).
// Least share, units: 64 streams of 2000 keys 59 with 32, 68 with 128; 8 is no
// faster, and a share of one unit a warp is no work.
constexpr int kMinShare = 32;
// Streams of at most this many units are not split: 8 of 1000 keys 12.6 with 64,
// 14.1 with 32; 64 of 1000 keys 39.5 and 42.2; 64 of 2000 keys 59.4 with 64, 61.5
// with 128.
constexpr int kWholeUnits = 64;
// Units (of one head) that a CTA's further segment costs, up to which slots beat
// equal shares: 8 streams of 1024 to 8192 keys 24.9 with 64, 30.4 with 0; 16 of 4096
// keys of 32 kv heads 97 with 64, 104 with 256.
constexpr int kSegment = 64;
// Side by side go twice as many heads, up to 2^kMaxSide, while a CTA's share holds
// kSideUnits units of each.  256 streams of 4096 keys of 32 kv heads: 1446 with one
// head, 1319 two, 1307 four, 1286 eight.  8 streams of 1024 to 8192 keys 24.9 with
// 128, 31.8 with 32; 64 of 2000 keys 59.4 with 128, 66.7 with 512.
constexpr int kMaxSide = 3, kSideUnits = 128;
// Rows per kv head up to which a sequence runs here; longer query blocks fill
// the 128-row tiles of the tcgen05 kernel, which takes as long for few rows as
// for 128 but is the slower to start and to join.  In us, here / there, on 4096
// keys of 8 kv heads (32 query heads), D = 128:
//   sequences   48 rows     64 rows     80 rows
//    4           30 / 49     37 / 48     51 / 48
//   16           97 / 103   115 / 102     - / 103
//   64          285 / 320   363 / 317   447 / 320
// and 64 sequences of 512 keys 88 / 77 with 48 rows, 109 / 75 with 64.
constexpr int kSmallRows = 64, kSmallRowsMany = 48;
constexpr int kManyStreams = 64;  // sequences x kv heads from which the second holds

template <int D>
struct Layout {
  static constexpr int kStages = D == 128 ? 6 : 12;        // units in a warp's ring
  static constexpr int kHalf = kKeys * D;                  // bytes of K (or V) in a stage
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kRing = kStages * kStage;           // of a warp
  static constexpr int kOffO = kWarps * kRing;             // float [kWarps][8 rows][D]
  static constexpr int kOffM = kOffO + kWarps * 8 * D * 4;
  static constexpr int kOffL = kOffM + kWarps * kRows * 4;
  static constexpr int kOffFlag = kOffL + kWarps * kRows * 4;
  static constexpr int kOffSums = kOffO;  // long long [kThreads + 3 kWarps], before the first merge
  static constexpr int kBytes = kOffFlag + 16;
  static_assert(kBytes <= 232448, "shared memory");
};

struct Seq {
  int q0, qlen, lk, units, tiles;  // tiles: 16-row tiles of a kv head
  int cost;                        // of one tile's stream: its units, or the slots it is cut into
  int chunk;                       // units of a slot (all of them where the cost counts units)
};

// `slot` > 0: streams are cut into slots of at most that many units.
__device__ __forceinline__ Seq load_seq(const AttendParams& p, int b, int slot, bool tell) {
  const SeqRows r = seq_rows(p, b, tell);
  Seq s{r.q0, r.qlen, r.lk, 0, 0, 0, 0};
  if ((long long)s.qlen * p.G > p.small_rows) s.qlen = 0;  // not this kernel's
  if (s.qlen == 0) return s;
  s.units = max(1, (s.lk + kKeys - 1) / kKeys);
  s.cost = s.chunk = s.units;
  if (slot > 0) {
    s.cost = (s.units - 1) / slot + 1;
    s.chunk = (s.units - 1) / s.cost + 1;
  }
  s.tiles = (s.qlen * p.G + kRows - 1) / kRows;
  return s;
}

// Cost of one kv head, or of one group of them, of the sequence.
__device__ __forceinline__ long long cost_of(const Seq& s) { return (long long)s.cost * s.tiles; }

// A position in a CTA's share: one segment (units [u, u + len) of a stream).
struct Cursor {
  int b, h, tile, u, len;  // h: group of neighbouring kv heads
  long long left;          // cost of the share from u on
  int groups;
  int slot;                // load_seq's
  Seq s;

  // Units of the segment that hold a key some row of the tile sees.
  __device__ __forceinline__ int seen(const AttendParams& p) const {
    if (!p.causal) return len;
    const int last = min((tile + 1) * kRows, s.qlen * p.G) - 1;
    const int end = min(s.lk, last / p.G + s.lk - s.qlen + 1);
    return min(len, max(0, (end + kKeys - 1) / kKeys - u));
  }
  __device__ __forceinline__ void next(const AttendParams& p) {
    left -= slot > 0 ? 1 : len;
    u = slot > 0 ? u + len : s.units;
    len = 0;
    if (left <= 0) return;
    if (u < s.units) {
      len = min(s.chunk, s.units - u);
      return;
    }
    u = 0;
    if (++tile == s.tiles) {
      tile = 0;
      if (++h == groups) {
        h = 0;
        do {
          if (++b >= p.B) {  // (lengths that change under the launch)
            left = 0;
            return;
          }
          s = load_seq(p, b, slot, false);
        } while (s.units == 0);
      }
    }
    len = slot > 0 ? s.chunk : (int)min((long long)s.units, left);
  }
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  const int n = take ? 16 : 0;  // 0: the slot is filled with zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Byte offset of 16-byte chunk c of row r (a key) in a stage.  D = 128: a row
// fills all banks; D = 64: two rows do.
template <int D>
__device__ __forceinline__ int slot_of(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ ((2 * (r & 3)) ^ (r & 4))) << 4);
  const int line = r >> 1;
  return line * 128 + (((((r & 1) << 2) | c) ^ (2 * (line & 3))) << 4);
}

// Key (of 16) of accumulator column j (0, 1) of key tile n (0, 1) in lane
// group position t.
template <int D>
__device__ __forceinline__ int key_of(int n, int j, int t) {
  return D == 128 ? 8 * n + t + 4 * j : 8 * n + 2 * t + j;
}

// Columns (bit hf D / 8 + e of x and y: column (2 t + hf) D / 8 + e) in which V
// has a NaN at one of the unit's first end0 (x), end1 (y) keys.
template <int D>
__device__ __noinline__ uint2 nan_columns(const uint8_t* sv, int t, int end0, int end1) {
  uint2 hit = make_uint2(0, 0);
  for (int i = 0; i < D / 4; ++i) {
    const int col = t * (D / 4) + i;
    for (int key = 0; key < kKeys; ++key) {
      if ((sv[slot_of<D>(key, col >> 4) + (col & 15)] & 0x7f) != 0x7f) continue;
      if (key < end0) hit.x |= 1u << i;
      if (key < end1) hit.y |= 1u << i;
    }
  }
  return hit;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__
                                                                 AttendParams p) {
  using L = Layout<D>;
  using E = Elem<T>;
  constexpr int kQ = D / 16;   // QK^T steps
  constexpr int kO = D / 8;    // PV column tiles; a lane holds columns [kO 2t, kO 2t + 2 kO)
  extern __shared__ __align__(128) uint8_t smem[];
  float* sO = reinterpret_cast<float*>(smem + L::kOffO);
  float* sM = reinterpret_cast<float*>(smem + L::kOffM);
  float* sL = reinterpret_cast<float*>(smem + L::kOffL);
  long long* sSums = reinterpret_cast<long long*>(smem + L::kOffSums);
  int* sFlag = reinterpret_cast<int*>(smem + L::kOffFlag);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;

  // ---- the CTA's share
  // Rolled loops: what runs once costs its instructions' way from L2, about a
  // dozen cycles each.  First the batch's running sums for one kv head, a thread
  // `per` sequences: units, tiles, and the longest stream.
  const int per = (p.B + kThreads - 1) / kThreads, ctas = (int)gridDim.x;
  int slot = 0, hw_log2 = 0, groups = p.Hkv, tiles = 0;
  long long total = 0, incl = 0;
  {
    int incl_t = 0, longest = 0;
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b >= p.B) break;
      const Seq s = load_seq(p, b, 0, blockIdx.x == 0);
      incl += cost_of(s);
      incl_t += s.tiles;
      longest = max(longest, s.units);
    }
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      const int z = __shfl_up_sync(0xffffffffu, incl_t, o);
      if (lane >= o) {
        incl += y;
        incl_t += z;
      }
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 31) {
      sSums[kThreads + warp] = incl;
      reinterpret_cast<int2*>(sM)[warp] = make_int2(incl_t, longest);
    }
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
      const long long x = sSums[kThreads + w];
      const int2 y = reinterpret_cast<const int2*>(sM)[w];
      if (w < warp) {
        incl += x;
        incl_t += y.x;
      }
      total += x;
      tiles += y.x;
      longest = max(longest, y.y);
    }
    if (longest <= kWholeUnits) {  // each stream one slot
      slot = kWholeUnits;
      incl = incl_t;
      total = tiles;
    } else {
      // Neighbouring kv heads side by side: 2^hw_log2 of them, each with 8 >>
      // hw_log2 of the warps, while a share stays long.
      while (hw_log2 < kMaxSide && (p.Hkv >> hw_log2) % 2 == 0 &&
             total * p.Hkv >= ((long long)kSideUnits << hw_log2) * ctas)
        ++hw_log2;
      groups = p.Hkv >> hw_log2;
    }
  }
  // How the streams are dealt.  Short ones whole.  A few long ones in slots, one
  // a CTA: of a length that half a slot a stream less fills the CTAs with, where
  // that suffices, or one that always does.  Otherwise equal shares that cut
  // streams anywhere -- every CTA is as long, but a segment more costs it what
  // kSegment units do.
  if (slot == 0 && tiles * (float)groups < ctas) {
    const float all = (float)(total * groups), streams = (float)(tiles * groups);
    const int most = (int)(all / ctas) + (kSegment >> hw_log2);
    int other = (int)(all / (ctas - streams)) + 2;  // always suffices
    slot = (int)(all / (ctas - 0.5f * streams)) + 2;
    if (slot > most) slot = 0;
#pragma unroll 1
    for (int pass = 1; slot > 0 || pass == 2; ++pass) {
      incl = 0;
#pragma unroll 1
      for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b < p.B) incl += cost_of(load_seq(p, b, slot, false));
      }
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) sSums[kThreads + pass * kWarps + warp] = incl;
      __syncthreads();
      total = 0;
#pragma unroll 1
      for (int w = 0; w < kWarps; ++w) {
        const long long x = sSums[kThreads + pass * kWarps + w];
        if (w < warp) incl += x;
        total += x;
      }
      if (pass == 2 || total * groups <= ctas) break;
      slot = other > most ? 0 : other;
    }
  }
  sSums[tid] = incl;
  __syncthreads();
  const int hw = 1 << hw_log2, step_u = kWarps >> hw_log2;
  const int my_u = warp & (step_u - 1), my_hh = warp >> (3 - hw_log2);
  total *= groups;
  long long share = quotient(total + gridDim.x - 1, gridDim.x);
  if (slot == 0) share = max((share + step_u - 1) & ~(long long)(step_u - 1), (long long)kMinShare);
  const long long first = share * blockIdx.x;
  if (first >= total) {
    griddep_wait();
    return;
  }
  Cursor at{};
  long long stream0;  // cost of the streams in front of the segment's
  {
    int lo = 0;  // the first thread whose sum passes `first`
    for (int step = kThreads / 2; step > 0; step >>= 1)
      if (sSums[lo + step - 1] * groups <= first) lo += step;
    long long off = first - (lo > 0 ? sSums[lo - 1] * groups : 0);
    at.groups = groups;
    at.slot = slot;
    at.b = lo * per;
    at.s = load_seq(p, at.b, slot, false);
    while (off >= cost_of(at.s) * groups && at.b + 1 < p.B) {
      off -= cost_of(at.s) * groups;
      at.s = load_seq(p, ++at.b, slot, false);
    }
    const long long head = cost_of(at.s);
    at.h = (int)quotient(off, head);
    const long long rest = off - at.h * head;
    at.tile = (int)quotient(rest, at.s.cost);
    at.u = (int)(rest - (long long)at.tile * at.s.cost);  // units, or slots, of the stream in front
    stream0 = first - at.u;
    if (slot > 0) at.u *= at.s.chunk;
    at.left = min(share, total - first);
    at.len = slot > 0 ? min(at.s.chunk, at.s.units - at.u)
                      : (int)min((long long)(at.s.units - at.u), at.left);
  }

  __syncthreads();  // sSums lies where the segments' results go

  // ---- the warp's copies: units my_u, my_u + step_u, ... of a segment
  constexpr int kChunks = D / 16, kRowsAt = 32 / kChunks;  // keys a warp copies at a time
  const int my_c = lane % kChunks, my_r = lane / kChunks;
  const uint32_t ring = smem_u32(smem) + warp * L::kRing;
  const int64_t k_lane = (int64_t)my_r * p.k_st + my_c * 16, v_lane = (int64_t)my_r * p.v_st + my_c * 16;
  const int64_t k_next = (int64_t)kRowsAt * p.k_st, v_next = (int64_t)kRowsAt * p.v_st;
  Cursor ahead = at;
  int a_i = my_u, a_seen = ahead.seen(p);
  // Table entries of the warp's next 32 units of the segment, one a lane, from
  // unit e_from on: one latency for all of them.
  int entries = 0, e_from = 0;
  const uint8_t *k_head = p.k_cache + (ahead.h * hw + my_hh) * p.k_sh + k_lane,
                *v_head = p.v_cache + (ahead.h * hw + my_hh) * p.v_sh + v_lane;
  const int32_t* a_row = p.block_table + (int64_t)ahead.b * p.bt_stride;
  auto read_entries = [&]() {
    e_from = a_i;
    const int i = a_i + lane * step_u;
    if (ahead.left > 0 && i < a_seen) entries = __ldg(a_row + ((ahead.u + i) >> p.page_shift));
  };
  auto find = [&]() {  // moves to the warp's next unit
    if (a_i < a_seen) {
      if (a_i == e_from + 32 * step_u) read_entries();
      return;
    }
    while (ahead.left > 0 && a_i >= a_seen) {
      ahead.next(p);
      if (ahead.left <= 0) return;
      a_i = my_u;
      a_seen = ahead.seen(p);
    }
    k_head = p.k_cache + (ahead.h * hw + my_hh) * p.k_sh + k_lane;
    v_head = p.v_cache + (ahead.h * hw + my_hh) * p.v_sh + v_lane;
    a_row = p.block_table + (int64_t)ahead.b * p.bt_stride;
    read_entries();
  };
  auto copy = [&](int stage) {
    if (ahead.left > 0) {
      const int unit = ahead.u + a_i;
      int page = __shfl_sync(0xffffffffu, entries, (a_i - e_from) >> (3 - hw_log2));
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0 && unit * kKeys < ahead.s.lk) report(p.err, PA_DEVERR_PAGE_OOB, ahead.b, unit);
        page = 0;
      }
      const int row0 = (unit & ((1 << p.page_shift) - 1)) * kKeys;
      const uint32_t dst = ring + stage * L::kStage;
      const uint8_t* ks = k_head + ((int64_t)page * p.k_sb + (int64_t)row0 * p.k_st);
      const uint8_t* vs = v_head + ((int64_t)page * p.v_sb + (int64_t)row0 * p.v_st);
      const int valid = ahead.s.lk - unit * kKeys;  // rows of the unit that hold a key
#pragma unroll
      for (int i = 0; i < kKeys / kRowsAt; ++i) {
        const int r = my_r + i * kRowsAt;
        const uint32_t to = dst + slot_of<D>(r, my_c);
        cp_async16(to, ks, r < valid);
        cp_async16(to + L::kHalf, vs, r < valid);
        ks += k_next;
        vs += v_next;
      }
      a_i += step_u;
      find();
    }
    cp_commit();  // an empty group where nothing is left keeps the count
  };
  // The raw query rows g and g + 8 of a segment's tile: read before the copies
  // of the first segment, or they wait behind all of them.
  // With them the head's scale.
  uint32_t raw[2][D / 64][8];
  float raw_scale = 1.f;
  auto read_rows = [&](const Cursor& w) {
    const int head = w.h * hw + my_hh, R = min(kRows, w.s.qlen * p.G - w.tile * kRows);
    if (p.k_scale != nullptr)
      asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(raw_scale) : "l"(p.k_scale + head));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // (rows behind the last are read as the tile's first, and cleared when used)
      const int row = w.tile * kRows + (g + 8 * j < R ? g + 8 * j : 0);
      const int i = row / p.G, h = head * p.G + row % p.G;
      const T* src = reinterpret_cast<const T*>(p.q) + (int64_t)(w.s.q0 + i) * p.q_st +
                     (int64_t)h * p.q_sh + t * 16;
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4 x = load16(src + c * 64 + e * 8);
          raw[j][c][4 * e] = x.x; raw[j][c][4 * e + 1] = x.y;
          raw[j][c][4 * e + 2] = x.z; raw[j][c][4 * e + 3] = x.w;
        }
    }
  };
  read_rows(at);
  if (a_i < a_seen)
    read_entries();
  else
    find();
#pragma unroll 1
  for (int i = 0; i < L::kStages; ++i) copy(i);
  int stage = 0;

  // ---- segments
  for (;;) {
    const int R = min(kRows, at.s.qlen * p.G - at.tile * kRows);
    const float ks = raw_scale;
    uint32_t qa[kQ][4];
    float f[2];  // score factor of rows g, g + 8 (log2 domain)
    int lim[2];  // keys they see
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = g + 8 * j;
      const int row = at.tile * kRows + r;
      const bool live = r < R;
      lim[j] = p.causal && live ? min(at.s.lk, row / p.G + at.s.lk - at.s.qlen + 1) : at.s.lk;
      uint32_t w[D / 64][8];
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) w[c][e] = live ? raw[j][c][e] : 0u;
      f[j] = fabsf(ks) * p.scale_log2;
      if constexpr (sizeof(T) == 2 && !std::is_same<T, __half>::value) {
        uint32_t top = 0;  // bits of the largest magnitude
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            top = max(top, max((w[c][e] & 0x7fffu) << 16, w[c][e] & 0x7fff0000u));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = (int)(top >> 23);  // biased exponent
        // 2^(127 - ex) scales the row to [1, 2) (to [2, 4) at the top of the
        // range); rows of zeros, of subnormals and rows with an infinity or
        // NaN stay as they are
        const bool turn = ex > 0 && ex < 255;
        const int by = min(ex, 253);
        const float down = turn ? __uint_as_float((uint32_t)(254 - by) << 23) : 1.f;
        if (turn) f[j] *= __uint_as_float((uint32_t)by << 23);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 x = E::to_f2(w[c][e]);
            w[c][e] = Elem<__half>::from_f2(x.x * down, x.y * down);
          }
      }
      const uint32_t flip = ks < 0.f ? 0x80008000u : 0u;
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          qa[c * 4 + e][j] = w[c][2 * e] ^ flip;
          qa[c * 4 + e][2 + j] = w[c][2 * e + 1] ^ flip;
        }
    }
    // every row of the tile sees the keys below this
    const int all = p.causal ? max(0, min(at.s.lk, at.tile * kRows / p.G + at.s.lk - at.s.qlen + 1))
                             : at.s.lk;
    float o[kO][4];
#pragma unroll
    for (int e = 0; e < kO; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[e][i] = 0.f;
    float m[2] = {neg_inf(), neg_inf()}, l[2] = {0.f, 0.f};  // m: the reference less kShift

    const int n = at.seen(p);
    // N of the warp's units at a time (two where there are two: twice the
    // independent work for the same waits): i, i + step_u.
    auto step = [&](auto units, int i) {
      constexpr int N = decltype(units)::value;
      cp_wait<L::kStages - N>();
      __syncwarp();  // every lane's copies of the units
      const uint8_t* sk[N];
#pragma unroll
      for (int u = 0; u < N; ++u) {
        int at_stage = stage + u;
        if (at_stage >= L::kStages) at_stage -= L::kStages;
        sk[u] = smem + warp * L::kRing + at_stage * L::kStage;
      }
      // S: c[2 u + nt] is key tile nt of unit u
      float c[2 * N][4];
#pragma unroll
      for (int x = 0; x < 2 * N; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[x][e] = 0.f;
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf) {
        uint4 x[2 * N];
#pragma unroll
        for (int y = 0; y < 2 * N; ++y) {
          // column g of the tile: the inverse of key_of
          const int key = D == 128 ? 8 * (y & 1) + (g >> 1) + 4 * (g & 1) : 8 * (y & 1) + g;
          x[y] = *reinterpret_cast<const uint4*>(sk[y >> 1] + slot_of<D>(key, hf * 4 + t));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int y = 0; y < 2 * N; ++y) {
            const uint32_t w[4] = {x[y].x, x[y].y, x[y].z, x[y].w};
            uint32_t b0, b1;
            f16x4_of(w[e], b0, b1);
            mma16816(c[y], qa[hf * 4 + e], b0, b1);
          }
      }
      // softmax
      const int key0 = (at.u + i) * kKeys, key_step = step_u * kKeys;  // unit u: key0 + u key_step
      const bool part = key0 + (N - 1) * key_step + kKeys > all;  // not seen whole by every row
      if (part) {
#pragma unroll
        for (int y = 0; y < 2 * N; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + (y >> 1) * key_step + key_of<D>(y & 1, e & 1, t) >= lim[e >> 1])
              c[y][e] = neg_inf();
      }
      float top[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        top[j] = fmaxf(c[0][2 * j], c[0][2 * j + 1]);
#pragma unroll
        for (int y = 1; y < 2 * N; ++y) top[j] = max3(top[j], c[y][2 * j], c[y][2 * j + 1]);
        top[j] *= f[j];
      }
      if (__any_sync(0xffffffffu,
                     top[0] > m[0] + (kShift + kSlack) || top[1] > m[1] + (kShift + kSlack))) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 1));
          top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 2));
          const float to = fmaxf(m[j], top[j] - kShift);
          const float by = m[j] == to ? 1.f : ex2(m[j] - to);
          m[j] = to;
          l[j] *= by;
#pragma unroll
          for (int e = 0; e < kO; ++e) {
            o[e][2 * j] *= by;
            o[e][2 * j + 1] *= by;
          }
        }
      }
      // a row that has seen no key yet has the reference -inf: 0 stands in
      const float m0 = m[0] == neg_inf() ? 0.f : m[0], m1 = m[1] == neg_inf() ? 0.f : m[1];
#pragma unroll
      for (int y = 0; y < 2 * N; ++y) {
        c[y][0] = ex2(fmaf(c[y][0], f[0], -m0));
        c[y][1] = ex2(fmaf(c[y][1], f[0], -m0));
        c[y][2] = ex2(fmaf(c[y][2], f[1], -m1));
        c[y][3] = ex2(fmaf(c[y][3], f[1], -m1));
      }
      if (part) {  // (a factor of zero turns -inf into NaN)
#pragma unroll
        for (int y = 0; y < 2 * N; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + (y >> 1) * key_step + key_of<D>(y & 1, e & 1, t) >= lim[e >> 1])
              c[y][e] = 0.f;
      }
      uint32_t pa[N][4];
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const float(&x)[4] = c[2 * u];
        const float(&y)[4] = c[2 * u + 1];
        l[0] += (x[0] + x[1]) + (y[0] + y[1]);
        l[1] += (x[2] + x[3]) + (y[2] + y[3]);
        pa[u][0] = Elem<__half>::from_f2(x[0], x[1]);
        pa[u][1] = Elem<__half>::from_f2(x[2], x[3]);
        pa[u][2] = Elem<__half>::from_f2(y[0], y[1]);
        pa[u][3] = Elem<__half>::from_f2(y[2], y[3]);
      }
      // O
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const uint8_t* sv = sk[u] + L::kHalf;
        constexpr int kWords = kO / 4;
        uint32_t v[4][kWords];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key_of<D>(e >> 1, e & 1, t);
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(sv + slot_of<D>(key, g));
            v[e][0] = x.x; v[e][1] = x.y; v[e][2] = x.z; v[e][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(sv + slot_of<D>(key, g >> 1) + (g & 1) * 8);
            v[e][0] = x.x; v[e][1] = x.y;
          }
        }
        if (part) {
          // A NaN in V at a key that only some rows see must not reach the
          // others through 0 x NaN: it is taken out of the product here and
          // put into the accumulators of the rows that do see it.
          uint32_t bad = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int w = 0; w < kWords; ++w) bad |= nan_bytes(v[e][w]);
          if (__any_sync(0xffffffffu, bad != 0)) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int w = 0; w < kWords; ++w) v[e][w] &= ~((nan_bytes(v[e][w]) >> 7) * 0xffu);
            const int k0 = key0 + u * key_step;
            const uint2 hit = nan_columns<D>(sv, t, min(lim[0] - k0, kKeys), min(lim[1] - k0, kKeys));
#pragma unroll
            for (int e = 0; e < kO; ++e) {
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                if ((hit.x >> (hf * kO + e)) & 1) o[e][hf] = __int_as_float(0x7fffffff);
                if ((hit.y >> (hf * kO + e)) & 1) o[e][2 + hf] = __int_as_float(0x7fffffff);
              }
            }
          }
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          const uint32_t x0 = __byte_perm(v[0][w], v[1][w], 0x5140);
          const uint32_t x1 = __byte_perm(v[2][w], v[3][w], 0x5140);
          const uint32_t y0 = __byte_perm(v[0][w], v[1][w], 0x7362);
          const uint32_t y1 = __byte_perm(v[2][w], v[3][w], 0x7362);
          uint32_t a0, a1, b0, b1;
          f16x4_of(x0, a0, a1);
          f16x4_of(x1, b0, b1);
          mma16816(o[4 * w], pa[u], a0, b0);
          mma16816(o[4 * w + 1], pa[u], a1, b1);
          f16x4_of(y0, a0, a1);
          f16x4_of(y1, b0, b1);
          mma16816(o[4 * w + 2], pa[u], a0, b0);
          mma16816(o[4 * w + 3], pa[u], a1, b1);
        }
      }
      __syncwarp();  // the stages have been read
#pragma unroll 1
      for (int u = 0; u < N; ++u) {
        copy(stage);
        stage = stage + 1 == L::kStages ? 0 : stage + 1;
      }
    };
    int i = my_u;
#pragma unroll 1
    for (; i + step_u < n; i += 2 * step_u) step(std::integral_constant<int, 2>{}, i);
    if (i < n) step(std::integral_constant<int, 1>{}, i);

    // ---- the warps' results: (m, l, O) of each, merged by column, eight rows
    // at a time
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      l[j] += __shfl_xor_sync(0xffffffffu, l[j], 1);
      l[j] += __shfl_xor_sync(0xffffffffu, l[j], 2);
      if (t == 0) {
        sM[warp * kRows + g + 8 * j] = m[j];
        sL[warp * kRows + g + 8 * j] = l[j];
      }
    }
    const bool done = at.u == 0 && at.len == at.s.units;  // not split
    const long long stream1 = stream0 + at.s.cost;
    const int slot = 2 * blockIdx.x + (at.u == 0 ? 1 : 0);
    constexpr int kChunksO = D / 4;
    auto write_row = [&](int hh, int r, int c, float4 x, float ref, float sum) {
      const int row = at.tile * kRows + r;
      const int i = row / p.G, h = (at.h * hw + hh) * p.G + row % p.G;
      const float vs = p.v_scale != nullptr ? __ldg(p.v_scale + at.h * hw + hh) : 1.f;
      const float by = sum == 0.f ? 0.f : vs / sum;  // NaN sums stay NaN
      T* dst = reinterpret_cast<T*>(p.out) + ((int64_t)(at.s.q0 + i) * p.Hq + h) * D + c * 4;
      uint2 y;
      y.x = E::from_f2(x.x * by, x.y * by);
      y.y = E::from_f2(x.z * by, x.w * by);
      *reinterpret_cast<uint2*>(dst) = y;
      if (c == 0 && p.lse != nullptr)
        p.lse[(int64_t)h * p.total_q + at.s.q0 + i] =
            sum == 0.f ? neg_inf() : (ref + log2f(sum)) * kLn2;
    };
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (8 * j >= R) break;
      if (j > 0) __syncthreads();  // the first eight rows have been read
      if (g + 8 * j < R) {
        float* dst = sO + (warp * 8 + g) * D;
#pragma unroll
        for (int q4 = 0; q4 < kO / 2; ++q4) {  // 16-byte chunks of the lane's 2 kO columns
          const int hf = q4 / (kO / 4), e = (q4 % (kO / 4)) * 4;
          const int c = t * (kO / 2) + q4;
          const int to = c ^ ((g & 1) | ((t << 1) & (D / 32 * 2 - 1)));
          *reinterpret_cast<float4*>(dst + to * 4) =
              make_float4(o[e][2 * j + hf], o[e + 1][2 * j + hf], o[e + 2][2 * j + hf],
                          o[e + 3][2 * j + hf]);
        }
      }
      __syncthreads();
      const int rows = min(R - 8 * j, 8);
#pragma unroll 1
      for (int x = tid; x < hw * rows * kChunksO; x += kThreads) {
        const int hr = x / kChunksO, c = x % kChunksO;
        const int hh = hr / rows, r = hr % rows, w0 = hh * step_u;  // the head's first warp
        const int from = c ^ ((r & 1) | (((c / (kO / 2)) << 1) & (D / 32 * 2 - 1)));
        const float* ms = sM + w0 * kRows + r + 8 * j;
        const float* ls = sL + w0 * kRows + r + 8 * j;
        const float* os = sO + (w0 * 8 + r) * D + from * 4;
        float ref = neg_inf();
        for (int w = 0; w < step_u; ++w) ref = fmaxf(ref, ms[w * kRows]);
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int w = 0; w < step_u; ++w) {
          const float mw = ms[w * kRows];
          const float by = mw == ref ? 1.f : ex2(mw - ref);
          const float4 y = *reinterpret_cast<const float4*>(os + w * 8 * D);
          sum = fmaf(by, ls[w * kRows], sum);
          acc.x = fmaf(by, y.x, acc.x);
          acc.y = fmaf(by, y.y, acc.y);
          acc.z = fmaf(by, y.z, acc.z);
          acc.w = fmaf(by, y.w, acc.w);
        }
        if (done) {
          write_row(hh, r + 8 * j, c, acc, ref, sum);
        } else {
          const int64_t to = ((int64_t)slot * kWarps + hh) * kRows + r + 8 * j;
          *reinterpret_cast<float4*>(p.part_o + to * D + c * 4) = acc;
          if (c == 0) p.part_ml[to] = make_float2(ref, sum);
        }
      }
    }
    if (!done) {
      const int cta0 = (int)quotient(stream0, share), cta1 = (int)quotient(stream1 - 1, share);
      __syncthreads();  // the partial rows of the CTA before its arrival
      if (tid == 0) {
        __threadfence();
        *sFlag = arrive_last(p.words + cta0, launch_tag(), cta1 - cta0 + 1) ? 1 : 0;
        __threadfence();
      }
      __syncthreads();
      if (*sFlag) {
        // A chunks of rows and C splits in flight a thread
        auto join = [&](auto rows_at_once, auto splits_at_once) {
          constexpr int A = decltype(rows_at_once)::value, C = decltype(splits_at_once)::value;
#pragma unroll 1
          for (int x0 = tid; x0 < hw * R * kChunksO; x0 += A * kThreads) {
            float ref[A], sum[A];
            float4 acc[A];
            int row[A];  // of a split's rows
            const int c = x0 % kChunksO;
#pragma unroll
            for (int k = 0; k < A; ++k) {
              const int hr = min((x0 + k * kThreads) / kChunksO, hw * R - 1);
              row[k] = (hr / R) * kRows + hr % R;
              ref[k] = neg_inf();
              sum[k] = 0.f;
              acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll 1
            for (int cta = cta0; cta <= cta1; cta += C) {
              float2 ml[C][A];
              float4 y[C][A];
#pragma unroll
              for (int j = 0; j < C; ++j) {
                const int s = min(cta + j, cta1);
                const int64_t from = (int64_t)(2 * s + (s == cta0 ? 1 : 0)) * kWarps * kRows;
#pragma unroll
                for (int k = 0; k < A; ++k) {
                  ml[j][k] = __ldcg(p.part_ml + from + row[k]);
                  y[j][k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + (from + row[k]) * D + c * 4));
                }
              }
#pragma unroll
              for (int j = 0; j < C; ++j) {
                if (cta + j > cta1) break;
#pragma unroll
                for (int k = 0; k < A; ++k) {
                  const float to = fmaxf(ref[k], ml[j][k].x);
                  const float b0 = ref[k] == to ? 1.f : ex2(ref[k] - to);
                  const float b1 = ml[j][k].x == to ? 1.f : ex2(ml[j][k].x - to);
                  ref[k] = to;
                  sum[k] = fmaf(b1, ml[j][k].y, sum[k] * b0);
                  acc[k].x = fmaf(b1, y[j][k].x, acc[k].x * b0);
                  acc[k].y = fmaf(b1, y[j][k].y, acc[k].y * b0);
                  acc[k].z = fmaf(b1, y[j][k].z, acc[k].z * b0);
                  acc[k].w = fmaf(b1, y[j][k].w, acc[k].w * b0);
                }
              }
            }
#pragma unroll
            for (int k = 0; k < A; ++k) {
              const int hr = (x0 + k * kThreads) / kChunksO;
              if (hr < hw * R) write_row(hr / R, hr % R, c, acc[k], ref[k], sum[k]);
            }
          }
        };
        if (hw * R * kChunksO <= kThreads)
          join(std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
        else
          join(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
      }
    }
    at.next(p);
    if (at.left <= 0) break;
    read_rows(at);
    if (at.u == 0) stream0 = stream1;
    __syncthreads();  // the merge has read what the next segment's overwrites
  }
  cp_wait<0>();
  // Launched behind the chunks' kernel this one may start before that one
  // ends; it must not end before it, for the stream's next kernel waits for
  // this one alone.
  griddep_wait();
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Workspace {
  size_t ml, o, chunk_words, chunk_ml, chunk_o, total;
};
Workspace workspace_of(int D, bool chunks) {
  const size_t ctas = (size_t)num_sms();
  Workspace w{};
  w.ml = align256(ctas * 8);
  w.o = w.ml + align256(ctas * 2 * kWarps * kRows * 8);
  w.total = w.o + align256(ctas * 2 * kWarps * kRows * D * 4);
  if (chunks) {
    w.chunk_words = w.total;
    w.chunk_ml = w.chunk_words + align256(ctas * 8);
    w.chunk_o = w.chunk_ml + align256(ctas * 2 * kChunkRows * 8);
    w.total = w.chunk_o + align256(ctas * 2 * kChunkRows * D * 4);
  }
  return w;
}

template <int D, typename T>
cudaError_t launch(const AttendParams& p, bool dependent, cudaStream_t st) {
  const int bytes = Layout<D>::kBytes;
  static std::atomic<uint64_t> devices{0};
  const cudaError_t e =
      allow_shared(reinterpret_cast<const void*>(attend_kernel<D, T>), bytes, &devices);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)num_sms());
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)bytes;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, attend_kernel<D, T>, p);
}

int small_rows(int B, int Hkv) {
  return (long long)B * Hkv >= kManyStreams ? kSmallRowsMany : kSmallRows;
}

// Whether a sequence of the call may have more rows per kv head than the
// warp-level kernel takes.
bool has_chunks(int B, int max_seqlen_q, int Hq, int Hkv) {
  return (long long)max_seqlen_q * (Hq / Hkv) > small_rows(B, Hkv);
}

bool aligned16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }

int check_cache8(const pa_tensor4& t, const char* name) {
  if (t.ptr == nullptr) return set_error(PA_ERR_INVALID_ARG, "%s.ptr is NULL", name);
  if (!aligned16(t.ptr) || t.stride_b <= 0 || t.stride_t <= 0 || t.stride_h <= 0 ||
      t.stride_b % 16 != 0 || t.stride_t % 16 != 0 || t.stride_h % 16 != 0)
    return set_error(PA_ERR_INVALID_ARG,
                     "%s must be 16-byte aligned with positive strides in multiples of 16 elements",
                     name);
  return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

PA_API size_t pa_fwd_varlen_e4m3_workspace_size(int B, int total_q, int max_seqlen_q, int Hq,
                                                int Hkv, int D, int max_seqlen_k) {
  (void)max_seqlen_k;
  if (B <= 0 || total_q <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0) return 0;
  return workspace_of(D, has_chunks(B, max_seqlen_q, Hq, Hkv)).total;
}

PA_API int pa_fwd_varlen_e4m3(const void* q, int64_t q_st, int64_t q_sh, pa_tensor4 k_cache,
                              pa_tensor4 v_cache, const float* k_scale, const float* v_scale,
                              const int32_t* cu_seqlens_q, const int32_t* seqlens_k,
                              const int32_t* block_table, int64_t bt_stride, int max_pages,
                              int page_size, int B, int total_q, int max_seqlen_q,
                              int max_seqlen_k, int Hq, int Hkv, int D, int64_t num_pages,
                              float scale, int causal, void* out, float* lse, void* workspace,
                              size_t workspace_bytes, int32_t* err_word, int dtype,
                              pa_stream_t stream) {
  if (dtype != PA_F16 && dtype != PA_BF16) return set_error(PA_ERR_UNSUPPORTED, "dtype %d", dtype);
  if (D != 64 && D != 128) return set_error(PA_ERR_UNSUPPORTED, "head_dim %d (64 or 128)", D);
  if (Hq < 1 || Hkv < 1) return set_error(PA_ERR_INVALID_ARG, "head counts must be >= 1");
  if (Hq % Hkv != 0)
    return set_error(PA_ERR_UNSUPPORTED, "Hq %d not a multiple of Hkv %d", Hq, Hkv);
  if (B < 0 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0)
    return set_error(PA_ERR_INVALID_ARG, "negative size argument");
  if (B == 0 || total_q == 0) return PA_OK;
  if (B > kMaxB) return set_error(PA_ERR_UNSUPPORTED, "more than %d sequences", kMaxB);
  int rc = 0;
  if ((rc = check_cache8(k_cache, "k_cache")) || (rc = check_cache8(v_cache, "v_cache"))) return rc;
  if (q == nullptr || out == nullptr || cu_seqlens_q == nullptr || seqlens_k == nullptr ||
      block_table == nullptr)
    return set_error(PA_ERR_INVALID_ARG,
                     "q, out, cu_seqlens_q, seqlens_k and block_table must be non-NULL");
  if (!aligned16(q) || !aligned16(out))
    return set_error(PA_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if (q_st <= 0 || q_sh <= 0 || q_st % 8 != 0 || q_sh % 8 != 0)
    return set_error(PA_ERR_INVALID_ARG, "q strides must be positive multiples of 8 elements");
  if (max_pages < 1 || bt_stride < max_pages || num_pages < 1)
    return set_error(PA_ERR_INVALID_ARG, "block table / pool sizes");
  if ((long long)total_q * (Hq / Hkv) > 0x7fffffff)
    return set_error(PA_ERR_UNSUPPORTED, "total_q * Hq / Hkv must be below 2^31");
  if (!(scale > 0.f) || !std::isfinite(scale))
    return set_error(PA_ERR_INVALID_ARG, "scale must be finite and > 0");
  AttendParams p{};
  p.page_shift = -1;
  for (int s = 0; s <= 4; ++s)
    if (page_size == kPage << s) p.page_shift = s;
  if (p.page_shift < 0)
    return set_error(PA_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
  if ((long long)max_pages * page_size > kMaxRowTokens)
    return set_error(PA_ERR_UNSUPPORTED, "a block table row must hold at most 2^31 - 4096 tokens");
  const bool chunks = has_chunks(B, max_seqlen_q, Hq, Hkv);
  if (chunks && ((long long)total_q * (Hq / Hkv) / kChunkRows + B) * (max_seqlen_k / 128 + 1) >
                    0x7fffffff)
    return set_error(PA_ERR_UNSUPPORTED, "total_q * Hq / Hkv * max_seqlen_k is too large");
  const Workspace ws = workspace_of(D, chunks);
  if (workspace == nullptr || workspace_bytes < ws.total)
    return set_error(PA_ERR_WORKSPACE, "workspace of %zu bytes required (got %zu)", ws.total,
                     workspace_bytes);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return set_error(PA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  uint8_t* wsb = reinterpret_cast<uint8_t*>(workspace);
  p.q = q;
  p.q_st = q_st; p.q_sh = q_sh;
  p.k_cache = reinterpret_cast<const uint8_t*>(k_cache.ptr);
  p.v_cache = reinterpret_cast<const uint8_t*>(v_cache.ptr);
  p.k_sb = k_cache.stride_b; p.k_st = k_cache.stride_t; p.k_sh = k_cache.stride_h;
  p.v_sb = v_cache.stride_b; p.v_st = v_cache.stride_t; p.v_sh = v_cache.stride_h;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.cu_seqlens_q = cu_seqlens_q;
  p.seqlens_k = seqlens_k;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.num_pages = num_pages;
  p.B = B;
  p.total_q = total_q;
  p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv;
  p.max_pages = max_pages;
  p.max_seqlen_k = max_seqlen_k;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = scale * kLog2e;
  p.out = out;
  p.lse = lse;
  p.err = err_word;
  // sequences of more rows than max_seqlen_q said run on the warp-level kernel
  p.small_rows = chunks ? small_rows(B, Hkv) : 0x7fffffff;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (chunks) {
    p.words = reinterpret_cast<unsigned long long*>(wsb + ws.chunk_words);
    p.part_ml = reinterpret_cast<float2*>(wsb + ws.chunk_ml);
    p.part_o = reinterpret_cast<float*>(wsb + ws.chunk_o);
    e = launch_chunks_e4m3(p, D, dtype, st);
    if (e != cudaSuccess)
      return set_error(PA_ERR_CUDA, "chunk launch: %s", cudaGetErrorString(e));
  }
  p.words = reinterpret_cast<unsigned long long*>(wsb);
  p.part_ml = reinterpret_cast<float2*>(wsb + ws.ml);
  p.part_o = reinterpret_cast<float*>(wsb + ws.o);
  if (dtype == PA_F16)
    e = D == 128 ? launch<128, __half>(p, chunks, st) : launch<64, __half>(p, chunks, st);
  else
    e = D == 128 ? launch<128, __nv_bfloat16>(p, chunks, st)
                 : launch<64, __nv_bfloat16>(p, chunks, st);
  if (e != cudaSuccess) return set_error(PA_ERR_CUDA, "attend launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

}  // extern "C"
