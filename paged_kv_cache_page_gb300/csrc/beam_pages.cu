// The pages of a beam search over a paged cache (sm_103a): block tables, lengths
// and pool after the beams have been replaced by their continuations
// (pa_beam_reorder), and the copies of the pages that several continuations
// would write to (pa_copy_pages).  flash-attention #824 and vLLM #6052 read K and
// V through block tables, so a beam's past is moved by moving table entries.
//
// Mathematics.  Child i of parent p_i has the parent's row of the table.  Beams
// branch off at a common length, so beams of a request share a page only at the
// same column of their rows, and everything about a page is decided by the K
// entries of its column, without reference counts:
//   - it is abandoned if no child's entry there is that page;
//   - a child's partly filled last page is copied if an earlier child has it too,
//     or another child has it as a whole page (which nobody will write to).
// Two sums over the batch (abandoned pages, copies) give each page its place on
// the stack of free pages and each copy its fresh page.
//
// One launch of one cluster of up to 16 CTAs, as the other calls of a step: the
// outputs may replace the inputs, and pages pushed by one request are popped by
// another, so all CTAs meet three times.  What bounds it is latency: loads of
// the table (a lane a column, the K entries of it in registers), the sums, the
// stores.  Every CTA gets the sums of every request and scans all of them.
//
// Measured: 5.3 us for one request of 4 beams, 6.4 for 32 of 5, 9.4 for 64 of 8.
//
// The copy moves (len mod page_size) tokens of k and v of every layer; it is
// bound by memory: 16 bytes a thread, four in flight.  5990 tokens of 8 caches, 2 KB
// each: 30.5 us, 6.4 TB/s.
#include <cooperative_groups.h>

#include <atomic>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kMaxBeams = 32;
constexpr int kMaxRows = 4096;
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = kMaxRows / kThreads;  // requests a thread scans
constexpr int kMaxCluster = 16;
constexpr int kMaxItems = 0x7fffffff - 0xffff;
constexpr uint32_t kAll = 0xffffffffu;

struct ReorderParams {
  const int32_t* parents;
  const int32_t* seqlens;
  const int32_t* table;
  int64_t bt_stride;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* table_out;
  int64_t bto_stride;
  int32_t* seqlens_out;
  int32_t* copies;
  int32_t* free_count_out;
  int32_t* err;
  int B, K, max_pages, page_log2, num_pages;
  int warps;  // of a request (a power of two)
};

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A load that sees what other threads of the cluster have stored.
__device__ __forceinline__ int load_l2(const int32_t* p) { return __ldcg(p); }

// The beams of a request, one a lane.
struct Beams {
  int len;     // tokens of beam `lane` (as given), and the pages they take
  int held;
  int parent;  // of child `lane`; -1: none
  int new_len, new_held;
  int partial;    // the child's partly filled column, or -1
  uint32_t used;  // beams that are a parent
  int columns;    // the largest held
  bool ok;        // (uniform) lengths and parents are sound
};
struct Given {  // of beam and child `lane`
  int len, parent;
};
__device__ __forceinline__ Given given_of(const ReorderParams& p, int g, int lane) {
  if (lane >= p.K) return {0, -1};
  return {p.seqlens[g * p.K + lane], p.parents[g * p.K + lane]};
}
__device__ __forceinline__ Beams beams_of(const ReorderParams& p, int g, int lane, Given given,
                                          bool rep) {
  Beams s;
  const int ps = 1 << p.page_log2;
  const long long cap = (long long)p.max_pages << p.page_log2;
  const int row = g * p.K + lane;
  s.len = given.len;
  s.parent = given.parent;
  const bool len_ok = s.len >= 0 && s.len <= cap;
  const bool par_ok = s.parent >= -1 && s.parent < p.K;
  if (rep && !len_ok) report(p.err, PA_DEVERR_LENGTH, row, s.len);
  if (rep && len_ok && !par_ok) report(p.err, PA_DEVERR_VALUE, row, s.parent);
  s.ok = __all_sync(kAll, len_ok && par_ok);
  s.held = len_ok ? (int)(((long long)s.len + ps - 1) >> p.page_log2) : 0;
  if (!par_ok) s.parent = -1;
  const int from = s.parent < 0 ? 0 : s.parent;
  const int len = __shfl_sync(kAll, s.len, from), held = __shfl_sync(kAll, s.held, from);
  s.new_len = s.parent < 0 ? 0 : len;
  s.new_held = s.parent < 0 ? 0 : held;
  s.partial = (s.new_len & (ps - 1)) && s.ok ? s.new_len >> p.page_log2 : -1;
  s.used = __reduce_or_sync(kAll, s.parent < 0 ? 0u : 1u << s.parent);
  s.columns = __reduce_max_sync(kAll, s.held);
  return s;
}

// The warp's part of the columns: whole multiples of 32.
struct Range {
  int begin, end;
};
__device__ __forceinline__ Range columns_of(int columns, int part, int parts) {
  const int each = (columns + 32 * parts - 1) / (32 * parts) * 32;
  return {min(columns, part * each), min(columns, (part + 1) * each)};
}

// The entries of column j: of the beams that hold it (a bit each), and the
// pages that no child holds there (the bit of the first beam that has one).
template <int KM>
struct Column {
  int e[KM];
  uint32_t held, gone;
};
template <int KM>
__device__ __forceinline__ void load_column(const ReorderParams& p, const Beams& s, int g, int j,
                                            Column<KM>& c) {
  const int32_t* row = p.table + (int64_t)g * p.K * p.bt_stride + j;
  c.held = 0;
#pragma unroll
  for (int k = 0; k < KM; ++k) {
    const int held = __shfl_sync(kAll, s.held, k);  // (0 behind the last beam)
    c.e[k] = -1;
    if (j < held) {
      c.e[k] = load_l2(row + k * p.bt_stride);
      c.held |= 1u << k;
    }
  }
  // prompt columns are one page for all beams
  bool alike = true;
  int first = -1;
#pragma unroll
  for (int k = KM - 1; k >= 0; --k)
    if (c.held >> k & 1) first = c.e[k];
#pragma unroll
  for (int k = 0; k < KM; ++k) alike = alike && (!(c.held >> k & 1) || c.e[k] == first);
  c.gone = c.held & s.used ? 0 : c.held & (0u - c.held);
  if (__all_sync(kAll, alike)) return;
  c.gone = 0;
#pragma unroll
  for (int k = 0; k < KM; ++k) {
    // beams with the page of beam k
    uint32_t same = 0;
#pragma unroll
    for (int q = 0; q < KM; ++q) same |= c.e[q] == c.e[k] ? 1u << q : 0u;
    same &= c.held;
    if ((same & s.used) == 0 && (same & (0u - same)) == 1u << k) c.gone |= 1u << k;
  }
}

// Whether child `lane` copies its last page, and that page (-1: it has no partly
// filled one).
__device__ __forceinline__ bool copies_page(const ReorderParams& p, const Beams& s, int g, int lane,
                                            int& page) {
  const int32_t* rows = p.table + (int64_t)g * p.K * p.bt_stride;
  const bool partly = s.partial >= 0;
  page = partly ? load_l2(rows + s.parent * p.bt_stride + s.partial) : -1;
  bool clash = false;
#pragma unroll 1
  for (int i = 0; i < p.K; ++i) {
    const int held = __shfl_sync(kAll, s.new_held, i), part = __shfl_sync(kAll, s.partial, i);
    const int par = __shfl_sync(kAll, s.parent, i);
    int other = __shfl_sync(kAll, page, i);  // child i's page in the lane's column, if that is its last
    if (!partly || i == lane || s.partial >= held) continue;
    if (part != s.partial) other = load_l2(rows + par * p.bt_stride + s.partial);
    else if (i > lane) continue;
    clash = clash || other == page;
  }
  return clash;
}

template <int KM>
__global__ void __launch_bounds__(kThreads) reorder_kernel(const ReorderParams p) {
  extern __shared__ int sm[];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = (int)blockDim.x;
  const int per = (p.B + ranks - 1) / ranks;             // requests of a CTA
  const int g0 = min(p.B, rank * per), g1 = min(p.B, g0 + per);
  int* s_given = sm;                   // [B] pages given back, then those in front
  int* s_taken = sm + p.B;             // [B] fresh pages, then those in front
  int* s_need = sm + 2 * p.B;          // [per] fresh pages of the CTA's requests
  int* s_part = s_need + per;          // [per][warps] pages given back by a warp's columns
  uint8_t* s_bad = reinterpret_cast<uint8_t*>(s_part + per * p.warps);  // [per]
  __shared__ int s_sums[2][32];
  __shared__ int s_fail, s_usable;
  __shared__ int s_usable_of[kMaxCluster];  // by CTA
  const int slots = threads / 32 / p.warps;  // requests at a time
  const int slot = warp / p.warps, part = warp % p.warps;

  cluster_arrive();  // (the others' shared memory is written once they have started)
  griddep_launch_dependents();
  for (int i = tid; i < per; i += threads) s_bad[i] = 0;
  for (int i = tid; i < 64; i += threads) s_sums[i >> 5][i & 31] = 0;
  if (tid == 0) {
    s_fail = p.B;
    s_usable = kMaxItems;
  }
  __syncthreads();
  griddep_wait();
  int free_now = load_l2(p.free_count);
  Given given0 = {0, -1};
  if (g0 + slot < g1) given0 = given_of(p, g0 + slot, lane);
  // The free pages that this call may take (no more than rows) are looked at while the
  // tables are read: the stack's usable part ends at an entry outside the pool.
  const int most = min(free_now < 0 ? 0 : min(free_now, p.num_pages), p.B * p.K);
  const int depth0 = rank * threads + tid;
  const int page0 = depth0 < most ? load_l2(p.free_pages + min(free_now, p.num_pages) - 1 - depth0) : 0;

  // Where a warp has one request it keeps what it has found out, and with 32 columns
  // at most loads nothing again.  (More requests than warps are a warp each.)
  const bool single = g0 + slot + slots >= g1;
  Beams s;
  Column<KM> c;
  Range r = {0, 0};
  int page = -1;  // the child's partly filled page
  bool copy = false;
  // ---- pages given back and fresh ones, request by request
#pragma unroll 1
  for (int g = g0 + slot; g < g1; g += slots) {
    s = beams_of(p, g, lane, g == g0 + slot ? given0 : given_of(p, g, lane), part == 0);
    r = {0, 0};
    int given = 0;
    if (s.ok) {
      r = columns_of(s.columns, part, p.warps);
#pragma unroll 1
      for (int j = r.begin + lane; j - lane < r.end; j += 32) {
        load_column<KM>(p, s, g, j < r.end ? j : 0x7fffffff, c);
        given += __popc(c.gone);
        uint32_t bad = 0;
#pragma unroll
        for (int k = 0; k < KM; ++k)
          if ((c.held >> k & 1) && (c.e[k] < 0 || c.e[k] >= p.num_pages)) bad |= 1u << k;
        if (bad) {
          report(p.err, PA_DEVERR_PAGE_OOB, g * p.K + __ffs((int)bad) - 1, j);
          s_bad[g - g0] = 1;
        }
      }
    } else if (lane == 0) {
      s_bad[g - g0] = 1;
    }
    given = __reduce_add_sync(kAll, given);
    if (lane == 0) s_part[(g - g0) * p.warps + part] = given;
    if (part == 0) {
      copy = s.ok && copies_page(p, s, g, lane, page);
      const int taken = __popc(__ballot_sync(kAll, copy));
      if (lane == 0) s_need[g - g0] = taken;
    }
  }
  if (free_now < 0 || free_now > p.num_pages) {
    if (rank == 0 && tid == 0) report(p.err, PA_DEVERR_CAPACITY, -1, free_now);
    free_now = free_now < 0 ? 0 : p.num_pages;
  }
  if (page0 < 0 || page0 >= p.num_pages) atomicMin(&s_usable, depth0);
#pragma unroll 1
  for (int i = depth0 + ranks * threads; i < most; i += ranks * threads) {
    const int e = load_l2(p.free_pages + free_now - 1 - i);
    if (e < 0 || e >= p.num_pages) atomicMin(&s_usable, i);
  }
  __syncthreads();
  cluster_wait();
  if (tid < ranks) cluster.map_shared_rank(s_usable_of, tid)[rank] = s_usable;
#pragma unroll 1
  for (int i = tid; i < (g1 - g0) * ranks; i += threads) {  // a request for a CTA
    const int g = i / ranks, to = i - g * ranks;
    int given = 0;
    for (int w = 0; w < p.warps; ++w) given += s_part[g * p.warps + w];
    cluster.map_shared_rank(s_given, to)[g0 + g] = s_bad[g] ? 0 : given;
    cluster.map_shared_rank(s_taken, to)[g0 + g] = s_bad[g] ? 0 : s_need[g];
  }
  cluster.sync();

  // ---- the sums in front of each request, and how far the pool goes
  const int room = p.num_pages - free_now;
  const int usable =
      min(free_now, __reduce_min_sync(kAll, lane < ranks ? s_usable_of[lane] : kMaxItems));
  int given[kPer], taken[kPer], my_given = 0, my_taken = 0;
  const int each = (p.B + threads - 1) / threads;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = tid * each + i;
    given[i] = taken[i] = 0;
    if (i < each && g < p.B) {
      given[i] = s_given[g];
      taken[i] = s_taken[g];
    }
    my_given += given[i];
    my_taken += taken[i];
  }
  int sum_given = my_given, sum_taken = my_taken;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kAll, sum_given, o), y = __shfl_up_sync(kAll, sum_taken, o);
    if (lane >= o) {
      sum_given += x;
      sum_taken += y;
    }
  }
  if (lane == 31) {
    s_sums[0][warp] = sum_given;
    s_sums[1][warp] = sum_taken;
  }
  __syncthreads();
  int at_given = sum_given - my_given + __reduce_add_sync(kAll, lane < warp ? s_sums[0][lane] : 0);
  int at_taken = sum_taken - my_taken + __reduce_add_sync(kAll, lane < warp ? s_sums[1][lane] : 0);
  const int all_given = __reduce_add_sync(kAll, s_sums[0][lane]);
  const int all_taken = __reduce_add_sync(kAll, s_sums[1][lane]);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = tid * each + i;
    if (i >= each || g >= p.B) continue;
    s_given[g] = at_given;
    s_taken[g] = at_taken;
    at_given += given[i];
    at_taken += taken[i];
    if (taken[i] > 0 && (long long)usable + min(at_given, room) < at_taken)
      atomicMin(&s_fail, g);
  }
  __syncthreads();
  const int fail = s_fail;  // requests [fail, B) stay as they are
  int top = all_given, used = all_taken;
  if (fail < p.B) {
    top = s_given[fail];
    used = s_taken[fail];
    if (rank == 0 && usable == free_now) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i < each && tid * each + i == fail) report(p.err, PA_DEVERR_CAPACITY, fail, taken[i]);
    }
  }
  if (top > room) {  // (pages that are in the tables and the pool twice)
    if (rank == 0 && tid == 0) report(p.err, PA_DEVERR_CAPACITY, -1, top);
    top = room;
  }
  top += free_now;

  // ---- abandoned pages onto the pool, children's entries
#pragma unroll 1
  for (int g = g0 + slot; g < g1; g += slots) {
    if (!single) {
      s = beams_of(p, g, lane, given_of(p, g, lane), false);
      copy = s.ok && copies_page(p, s, g, lane, page);
    }
    const bool moved = g < fail && !s_bad[g - g0];
    if (g == fail && usable < free_now && part == 0) {  // a page outside the pool stopped it
      const uint32_t first = __ballot_sync(kAll, copy);
      if (lane == __ffs((int)first) - 1) report(p.err, PA_DEVERR_PAGE_OOB, g * p.K + lane, s.partial);
    }
    int parent = s.parent, new_held = s.new_held;
    if (!moved) {  // every beam stays itself
      parent = lane < p.K ? lane : -1;
      new_held = s.held;
    }
    const bool held = single && s.ok && r.end - r.begin <= 32;  // the columns are in registers
    r = columns_of(s.columns, part, p.warps);
    int at = s_given[g];
    for (int i = 0; i < part; ++i) at += s_part[(g - g0) * p.warps + i];
#pragma unroll 1
    for (int j = r.begin + lane; j - lane < r.end; j += 32) {
      const int col = j < r.end ? j : 0x7fffffff;
      if (!held) load_column<KM>(p, s, g, col, c);
      if (moved) {
        const int mine = __popc(c.gone);
        if (__any_sync(kAll, mine != 0)) {
          int upto = mine;
#pragma unroll 1
          for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kAll, upto, o);
            if (lane >= o) upto += x;
          }
          int to = at + upto - mine;
          for (uint32_t left = c.gone; left != 0; left &= left - 1) {
            const int k = __ffs((int)left) - 1;
            int e = c.e[0];
#pragma unroll
            for (int q = 1; q < KM; ++q) e = q == k ? c.e[q] : e;
            if (to < room) p.free_pages[free_now + to] = e;
            ++to;
          }
          at += __shfl_sync(kAll, upto, 31);
        }
      }
      // (all of the column has been read before any of it is written)
#pragma unroll
      for (int i = 0; i < KM; ++i) {
        const int par = __shfl_sync(kAll, parent, i), end = __shfl_sync(kAll, new_held, i);
        if (col < end && !(par == i && p.table == p.table_out)) {
          int e = c.e[0];
#pragma unroll
          for (int q = 1; q < KM; ++q) e = q == par ? c.e[q] : e;
          p.table_out[((int64_t)g * p.K + i) * p.bto_stride + col] = e;
        }
      }
    }
    if (!single && lane < p.K) p.copies[3 * (g * p.K + lane)] = moved && copy ? page : -1;
  }
  cluster.sync();

  // ---- fresh pages, copies, lengths
  if (rank == 0 && tid == 0) *p.free_count_out = max(0, top - used);
#pragma unroll 1
  for (int g = g0 + slot; g < g1; g += slots) {
    if (part != 0) continue;
    const bool moved = g < fail && !s_bad[g - g0];
    const int row = g * p.K + lane;
    if (!single) {
      s = beams_of(p, g, lane, given_of(p, g, lane), false);
      page = lane < p.K ? load_l2(p.copies + 3 * row) : -1;
      copy = page >= 0;
    }
    int src = -1, dst = -1, tokens = 0;
    if (moved && __any_sync(kAll, copy)) {
      // fresh pages by column, then by child
      int before = 0;
#pragma unroll 1
      for (int i = 0; i < p.K; ++i) {
        const int part_i = __shfl_sync(kAll, s.partial, i);
        const bool copy_i = __shfl_sync(kAll, (int)copy, i) != 0;
        if (copy_i && (part_i < s.partial || (part_i == s.partial && i < lane))) ++before;
      }
      if (copy) {
        src = page;
        dst = load_l2(p.free_pages + top - 1 - (s_taken[g] + before));
        tokens = s.new_len & ((1 << p.page_log2) - 1);
        p.table_out[(int64_t)row * p.bto_stride + s.partial] = dst;
      }
    }
    if (lane < p.K) {
      p.copies[3 * row] = src;
      p.copies[3 * row + 1] = dst;
      p.copies[3 * row + 2] = tokens;
      p.seqlens_out[row] = moved ? s.new_len : s.len;
    }
  }
}

template <int KM>
cudaError_t launch_reorder(ReorderParams p, cudaStream_t st) {
  static std::atomic<uint64_t> asked{0}, wide{0}, allowed{0};
  // A warp for each 32 columns as far as they go, and as many CTAs of eight warps as
  // that fills (barriers of few warps are short); then larger ones.
  const int chunks = (p.max_pages + 31) / 32;
  int ctas = 1;
  while (ctas < kMaxCluster && ctas < p.B && (long long)p.B * chunks > (long long)ctas * 8) ctas *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cudaLaunchAttribute attrs[2] = {};
  cudaLaunchAttribute& at = attrs[0];
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  overlap_launch(&attrs[1]);
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  auto shape = [&] {
    const int per = (p.B + ctas - 1) / ctas;
    p.warps = 1;
    while (p.warps < kWarps && p.warps < chunks && p.warps * 2 * per <= kWarps) p.warps *= 2;
    const int warps = per * p.warps < 4 ? 4 : per * p.warps < kWarps ? per * p.warps : kWarps;
    cfg.blockDim = dim3((unsigned)(warps + p.warps - 1) / p.warps * p.warps * 32);
    cfg.dynamicSmemBytes = (size_t)p.B * 8 + (size_t)per * (p.warps + 1) * 4 + (size_t)per;
    cfg.gridDim = dim3((unsigned)ctas);
    at.val.clusterDim.x = (unsigned)ctas;
  };
  // 8 B a request, and of a CTA 4 B a warp's part (kWarps at most, or one a request), 4 B
  // and a flag a request
  const int most = kMaxRows * (8 + 4 + 4 + 1);
  cudaError_t e = allow_shared(reinterpret_cast<const void*>(reorder_kernel<KM>), most, &allowed);
  if (e != cudaSuccess) return e;
  shape();
  if (ctas > 8 &&
      !wide_clusters(reorder_kernel<KM>, kMaxCluster, kThreads, most, &asked, &wide)) {
    ctas = 8;
    shape();
  }
  return cudaLaunchKernelEx(&cfg, reorder_kernel<KM>, p);
}

// ------------------------------------------------------------------ copies
constexpr int kCopyThreads = 256;
constexpr int kMaxCaches = 256;

struct CopyParams {
  void* caches[kMaxCaches];
  const int32_t* copies;
  int64_t stride_b, stride_t, stride_h;  // bytes
  int n, n_caches, head_vecs, token_vecs, page_size, num_pages;
  int linear;  // the tokens of a page follow one another without gaps
  int32_t* err;
};

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int entry = blockIdx.x;
  const int32_t* copy = p.copies + 3 * (int64_t)entry;
  const int src = copy[0], dst = copy[1], tokens = copy[2];
  if (src < 0 || dst < 0 || tokens == 0) return;
  const bool first = blockIdx.y == 0 && threadIdx.x == 0;
  if (src >= p.num_pages || dst >= p.num_pages) {
    if (first) report(p.err, PA_DEVERR_PAGE_OOB, entry, src >= p.num_pages ? src : dst);
    return;
  }
  if (tokens < 0 || tokens > p.page_size) {
    if (first) report(p.err, PA_DEVERR_LENGTH, entry, tokens);
    return;
  }
  const int vecs = tokens * p.token_vecs;
  auto place = [&](int i) -> int64_t {
    if (p.linear) return (int64_t)i * 16;
    const int t = i / p.token_vecs, r = i - t * p.token_vecs, h = r / p.head_vecs;
    return t * p.stride_t + h * p.stride_h + (int64_t)(r - h * p.head_vecs) * 16;
  };
  for (int c = blockIdx.y; c < p.n_caches; c += gridDim.y) {
    const char* from = reinterpret_cast<const char*>(p.caches[c]) + src * p.stride_b;
    char* to = reinterpret_cast<char*>(p.caches[c]) + dst * p.stride_b;
    for (int i = threadIdx.x; i < vecs; i += 4 * kCopyThreads) {
      uint4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j * kCopyThreads < vecs)
          x[j] = __ldcs(reinterpret_cast<const uint4*>(from + place(i + j * kCopyThreads)));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j * kCopyThreads < vecs)
          *reinterpret_cast<uint4*>(to + place(i + j * kCopyThreads)) = x[j];
    }
  }
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

PA_API int pa_beam_reorder(const int32_t* parents, const int32_t* seqlens, int B, int K,
                           const int32_t* block_table, int64_t bt_stride, int max_pages,
                           int page_size, int32_t* free_pages, const int32_t* free_count,
                           int64_t num_pages, int32_t* block_table_out, int64_t bto_stride,
                           int32_t* seqlens_out, int32_t* copies, int32_t* free_count_out,
                           int32_t* err_word, pa_stream_t stream) {
  ReorderParams p{};
  if (B < 0 || K < 1) return set_error(PA_ERR_INVALID_ARG, "B must be >= 0 and K >= 1");
  if (K > kMaxBeams) return set_error(PA_ERR_UNSUPPORTED, "more than %d beams", kMaxBeams);
  if ((long long)B * K > kMaxRows)
    return set_error(PA_ERR_UNSUPPORTED, "more than %d rows", kMaxRows);
  if (max_pages < 1 || bt_stride < max_pages || bto_stride < max_pages)
    return set_error(PA_ERR_INVALID_ARG, "block tables need max_pages >= 1 and strides >= max_pages");
  if (num_pages < 1 || num_pages > kMaxItems)
    return set_error(PA_ERR_INVALID_ARG, "num_pages must be in [1, 2^31 - 2^16]");
  p.page_log2 = -1;
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) p.page_log2 = s;
  if (p.page_log2 < 0)
    return set_error(PA_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
  if (((long long)max_pages << p.page_log2) > kMaxRowTokens)
    return set_error(PA_ERR_UNSUPPORTED, "a block table row must hold at most 2^31 - 4096 tokens");
  // (every held entry may be given back: their number fits in 32 bits)
  if ((long long)B * K * max_pages > kMaxItems)
    return set_error(PA_ERR_UNSUPPORTED, "block tables of more than 2^31 - 2^16 entries");
  if (free_count == nullptr || free_count_out == nullptr || free_pages == nullptr)
    return set_error(PA_ERR_INVALID_ARG,
                     "free_pages, free_count and free_count_out must be non-NULL");
  if (B > 0 && (parents == nullptr || seqlens == nullptr || block_table == nullptr ||
                block_table_out == nullptr || seqlens_out == nullptr || copies == nullptr))
    return set_error(PA_ERR_INVALID_ARG,
                     "parents, seqlens, block_table, block_table_out, seqlens_out and copies must "
                     "be non-NULL");
  if (block_table == block_table_out && bt_stride != bto_stride)
    return set_error(PA_ERR_INVALID_ARG, "a table that is replaced keeps its stride");
  p.parents = parents;
  p.seqlens = seqlens;
  p.table = block_table;
  p.bt_stride = bt_stride;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.table_out = block_table_out;
  p.bto_stride = bto_stride;
  p.seqlens_out = seqlens_out;
  p.copies = copies;
  p.free_count_out = free_count_out;
  p.err = err_word;
  p.B = B;
  p.K = K;
  p.max_pages = max_pages;
  p.num_pages = (int)num_pages;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = K <= 4    ? launch_reorder<4>(p, st)
                        : K <= 8  ? launch_reorder<8>(p, st)
                        : K <= 16 ? launch_reorder<16>(p, st)
                                  : launch_reorder<32>(p, st);
  if (e != cudaSuccess) return set_error(PA_ERR_CUDA, "reorder launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

PA_API int pa_copy_pages(const int32_t* copies, int n, void* const* caches, int n_caches,
                         int64_t stride_b, int64_t stride_t, int64_t stride_h, int head_bytes,
                         int H, int page_size, int64_t num_pages, int32_t* err_word,
                         pa_stream_t stream) {
  if (n < 0 || n_caches < 0) return set_error(PA_ERR_INVALID_ARG, "negative n or n_caches");
  if (H < 1 || page_size < 1 || num_pages < 1)
    return set_error(PA_ERR_INVALID_ARG, "H, page_size and num_pages must be >= 1");
  if (num_pages > kMaxItems)
    return set_error(PA_ERR_UNSUPPORTED, "more than 2^31 - 2^16 pages");
  if (head_bytes < 16 || head_bytes % 16 != 0 || stride_b <= 0 || stride_b % 16 != 0 ||
      stride_t <= 0 || stride_t % 16 != 0 || stride_h <= 0 || stride_h % 16 != 0)
    return set_error(PA_ERR_INVALID_ARG,
                     "head_bytes and the strides must be positive multiples of 16");
  if ((long long)page_size * H * (head_bytes / 16) > (1 << 30))
    return set_error(PA_ERR_UNSUPPORTED, "a page of more than 2^34 bytes");
  if (n == 0 || n_caches == 0) return PA_OK;
  if (copies == nullptr || caches == nullptr)
    return set_error(PA_ERR_INVALID_ARG, "copies and caches must be non-NULL");
  for (int i = 0; i < n_caches; ++i)
    if (caches[i] == nullptr || reinterpret_cast<uintptr_t>(caches[i]) % 16 != 0)
      return set_error(PA_ERR_INVALID_ARG, "caches[%d] must be non-NULL and 16-byte aligned", i);
  CopyParams p;
  p.copies = copies;
  p.stride_b = stride_b;
  p.stride_t = stride_t;
  p.stride_h = stride_h;
  p.n = n;
  p.head_vecs = head_bytes / 16;
  p.token_vecs = H * p.head_vecs;
  p.page_size = page_size;
  p.num_pages = (int)num_pages;
  p.linear = (H == 1 || stride_h == head_bytes) &&
             (page_size == 1 || stride_t == (int64_t)H * head_bytes);
  p.err = err_word;
  for (int at = 0; at < n_caches; at += kMaxCaches) {
    p.n_caches = n_caches - at < kMaxCaches ? n_caches - at : kMaxCaches;
    for (int i = 0; i < p.n_caches; ++i) p.caches[i] = caches[at + i];
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)n, (unsigned)p.n_caches);
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr{};
    overlap_launch(&attr);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, copy_kernel, p);
    if (e != cudaSuccess) return set_error(PA_ERR_CUDA, "copy launch: %s", cudaGetErrorString(e));
  }
  return PA_OK;
}

}  // extern "C"
