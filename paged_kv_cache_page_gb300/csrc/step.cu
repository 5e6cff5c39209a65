// The bookkeeping of a serving step on the GPU (sm_103a): pages for the new
// tokens out of a pool of free pages, block tables, and each new token's slot
// and position (pa_plan_step); and pages given back to the pool
// (pa_release_pages).  vLLM #6052 "Unify the kernel used in flash attention
// backend" builds this metadata on the host for every step (block_tables,
// cumulative query lengths padded with repeated entries, slots for the cache
// write of vLLM #3010 "Introduce flash-attn"); here the lengths never leave
// the GPU, so a captured step needs no host work.
//
// Mathematics.  pages(x) = ceil(x / page_size); request b, with c_b tokens in
// the cache and n_b new ones, needs pages(c_b + n_b) - pages(c_b) pages.  Two
// inclusive sums over the batch -- needed pages and new tokens -- decide who
// is admitted: sums only grow, so "both fit" is a prefix of the batch, and the
// sums in front of an admitted request are already its offsets into the pool
// and into the packed rows.  One scan serves both.
//
// Both kernels are one launch of one cluster of up to 16 CTAs.  What bounds
// them is latency, not bytes (a step of 1024 requests moves 0.8 MB): a chain
// of launch, length loads, scan, binary search, table load, store -- and of
// instruction fetches: code that runs once comes from far away, and unrolled
// eight-fold, with eight searches side by side, the same steps took half as long
// again (64 requests now 3.8 us, 1024 with 33000 new tokens 8.9).  Every CTA
// of the cluster repeats the scan of the whole batch (at most 4096 entries,
// four a thread), which costs less than a second launch or a wait on another
// CTA's sums; the rows and pages are then dealt over the cluster's threads.
// A cluster and not a grid, because the outputs may replace the inputs
// (free_count_out = free_count, seqlens_k = cache_seqlens): the cluster's
// barrier tells when every CTA has read them.
#include <cooperative_groups.h>

#include <atomic>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace cg = cooperative_groups;

namespace pa {
int set_error(int code, const char* fmt, ...);

namespace {

constexpr int kThreads = 1024;
constexpr int kMaxB = 4096;
constexpr int kPer = kMaxB / kThreads;  // consecutive entries of the batch a thread scans
constexpr int kAtOnce = 4;
constexpr int kMaxItems = 0x7fffffff - 0xffff;  // pages, rows: dealt to warps in 32-bit places
constexpr int kCluster = 16;             // CTAs of the cluster at most (8 where 16 do not fit)

struct PlanParams {
  const int32_t* cache_seqlens;
  const int32_t* q_lens;
  int32_t* block_table;
  int64_t bt_stride;
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* cu_seqlens_q;
  int32_t* seqlens_k;
  int64_t* slots;
  int32_t* positions;
  int32_t* free_count_out;
  int32_t* err;
  int B, max_pages, page_log2, token_capacity;
  int num_pages;
};

struct ReleaseParams {
  const int32_t* cache_seqlens;
  const int32_t* keep_lens;
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* seqlens_out;
  int32_t* free_count_out;
  int32_t* err;
  int B, max_pages, page_log2;
  int num_pages;
};

// A load that stays where it is written (see load16).
__device__ __forceinline__ int load4(const int32_t* src) {
  int x;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(x) : "l"(src) : "memory");
  return x;
}

// Inclusive sums over the CTA of one 64-bit value a thread; `warp_sums` holds
// 32 values.
__device__ __forceinline__ long long block_scan(long long x, long long* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  // every warp sums the totals of the warps in front of it
  long long before = lane < warp ? warp_sums[lane] : 0;  // (warp < warps of the CTA)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  return x + before;
}

// The last b < n, from `b` on, with first[b] <= k, for ascending first[0] = 0
// (entries that hold nothing share their successor's start, so the one found
// holds k).  Most steps stay in the entry they came from.
__device__ __noinline__ int find_entry(const int* first, int n, int b, int k) {
  if (b + 1 >= n || first[b + 1] > k) return b;
  for (int step = 1 << (31 - __clz(n)); step > 0; step >>= 1)
    if (b + step < n && first[b + step] <= k) b += step;
  return b;
}

// The part of [0, n) that the warp handles: whole multiples of 32.
struct Range {
  int begin, end;
};
__device__ __forceinline__ Range warp_range(int n, int rank, int ranks) {
  const int warps = (int)blockDim.x / 32 * ranks;
  const int w = rank * ((int)blockDim.x / 32) + (int)threadIdx.x / 32;
  const int each = (n + 32 * warps - 1) / (32 * warps) * 32;
  return {min(n, w * each), min(n, (w + 1) * each)};
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanParams p) {
  extern __shared__ int sm[];
  int* s_row = sm;                // [B] first packed row of the entry
  int* s_page = sm + p.B;         // [B] first needed page of the entry
  int* s_old = sm + 2 * p.B;      // [B] tokens in the cache
  __shared__ long long s_sums[2][32];
  __shared__ int s_total[2];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x;
  const int ps = 1 << p.page_log2;
  const long long cap = (long long)p.max_pages << p.page_log2;

  int free_now = *p.free_count;
  if (free_now < 0 || free_now > p.num_pages) {
    if (rank == 0 && tid == 0) report(p.err, PA_DEVERR_CAPACITY, -1, free_now);
    free_now = free_now < 0 ? 0 : p.num_pages;
  }
  if (tid < 2) s_total[tid] = 0;

  // the thread's entries and their sums
  const int per = (p.B + (int)blockDim.x - 1) / (int)blockDim.x;
  int old[kPer], add[kPer], need[kPer];
  long long pages = 0, rows = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * per + i;
    old[i] = add[i] = need[i] = 0;
    if (i >= per || b >= p.B) continue;
    const int c = p.cache_seqlens[b], n = p.q_lens[b];
    const bool c_ok = c >= 0 && c <= cap;
    const bool ok = c_ok && n >= 0 && (long long)c + n <= cap;
    if (!ok && rank == 0) report(p.err, PA_DEVERR_LENGTH, b, c_ok ? n : c);
    old[i] = c;  // (kept as it is where it is malformed: the entry holds no page or row)
    add[i] = ok ? n : 0;
    if (ok) need[i] = ((c + n + ps - 1) >> p.page_log2) - ((c + ps - 1) >> p.page_log2);
    pages += need[i];
    rows += add[i];
  }
  long long pages_at = block_scan(pages, s_sums[0]) - pages;
  long long rows_at = block_scan(rows, s_sums[1]) - rows;

  // admission: a prefix of the batch
  int my_rows = 0, my_pages = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * per + i;
    if (i >= per || b >= p.B) continue;
    const bool before = pages_at <= free_now && rows_at <= p.token_capacity;
    const bool fits = pages_at + need[i] <= free_now && rows_at + add[i] <= p.token_capacity;
    if (before && !fits && rank == 0) report(p.err, PA_DEVERR_CAPACITY, b, need[i]);
    // (a refused entry keeps sums beyond every index that is looked up)
    s_row[b] = (int)min(rows_at, 0x7fffffffll);
    s_page[b] = (int)min(pages_at, 0x7fffffffll);
    s_old[b] = old[i];
    pages_at += need[i];
    rows_at += add[i];
    if (!fits) add[i] = 0;
    if (fits) {
      my_rows = (int)rows_at;
      my_pages = (int)pages_at;
    }
  }
  __syncthreads();  // s_total at zero, entries written
  my_rows = __reduce_max_sync(0xffffffffu, my_rows);
  my_pages = __reduce_max_sync(0xffffffffu, my_pages);
  if ((tid & 31) == 0) {
    atomicMax(&s_total[0], my_rows);
    atomicMax(&s_total[1], my_pages);
  }
  cluster.sync();  // totals; and every CTA has read the lengths and the count
  const int T = s_total[0], N = s_total[1];

  if (rank == 0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * per + i;
      if (i >= per || b >= p.B) continue;
      p.cu_seqlens_q[b] = min(s_row[b], T);
      p.seqlens_k[b] = old[i] + add[i];
    }
    if (tid == 0) {
      p.cu_seqlens_q[p.B] = T;
      *p.free_count_out = free_now - N;
    }
  }
  // A warp's pages and rows are neighbours, so its entries are found by a look
  // at the next one, and its loads and stores are whole lines.
  const int lane = tid & 31;
  Range r = warp_range(N, rank, ranks);
  for (int k = r.begin + lane, b = 0; k < r.end; k += 32) {
    b = find_entry(s_page, p.B, b, k);
    const int page = p.free_pages[free_now - 1 - k];
    const int j = ((s_old[b] + ps - 1) >> p.page_log2) + k - s_page[b];
    if (page < 0 || page >= p.num_pages) report(p.err, PA_DEVERR_PAGE_OOB, b, j);
    p.block_table[(int64_t)b * p.bt_stride + j] = page;
  }
  r = warp_range(p.token_capacity, rank, ranks);
  for (int t = r.begin + lane, b = 0; t < r.end; t += 32) {
    int64_t slot = -1;
    int pos = 0;
    if (t < T) {
      b = find_entry(s_row, p.B, b, t);
      const int c = s_old[b];
      pos = c + t - s_row[b];
      const int j = pos >> p.page_log2;
      const int fresh = j - ((c + ps - 1) >> p.page_log2);
      const int page = *(fresh >= 0 ? p.free_pages + (free_now - 1 - (s_page[b] + fresh))
                                    : p.block_table + ((int64_t)b * p.bt_stride + j));
      if (page >= 0 && page < p.num_pages)
        slot = ((int64_t)page << p.page_log2) + (pos & (ps - 1));
      else
        report(p.err, PA_DEVERR_PAGE_OOB, b, j);
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
}

__global__ void __launch_bounds__(kThreads) release_kernel(const ReleaseParams p) {
  extern __shared__ int sm[];
  int* s_at = sm;             // [B] the entry's first place among the released pages
  int* s_from = sm + p.B;     // [B] its first released table column
  __shared__ long long s_sums[32];
  __shared__ int s_total, s_bad;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x;
  const int ps = 1 << p.page_log2;
  const long long cap = (long long)p.max_pages << p.page_log2;

  int free_now = *p.free_count;
  if (free_now < 0 || free_now > p.num_pages) {
    if (rank == 0 && tid == 0) report(p.err, PA_DEVERR_CAPACITY, -1, free_now);
    free_now = free_now < 0 ? 0 : p.num_pages;
  }
  if (tid == 0) s_total = s_bad = 0;

  const int per = (p.B + (int)blockDim.x - 1) / (int)blockDim.x;
  int len[kPer], keep[kPer], gone[kPer];
  long long sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * per + i;
    len[i] = keep[i] = gone[i] = 0;
    if (i >= per || b >= p.B) continue;
    len[i] = p.cache_seqlens[b];
    keep[i] = min(p.keep_lens[b], len[i]);
    const bool len_ok = len[i] >= 0 && len[i] <= cap;
    if (!len_ok || keep[i] < 0) {
      if (rank == 0) report(p.err, PA_DEVERR_LENGTH, b, len_ok ? keep[i] : len[i]);
      keep[i] = len[i];
    } else {
      gone[i] = ((len[i] + ps - 1) >> p.page_log2) - ((keep[i] + ps - 1) >> p.page_log2);
    }
    sum += gone[i];
  }
  long long at = block_scan(sum, s_sums) - sum;
  const int room = p.num_pages - free_now;
  int my_total = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * per + i;
    if (i >= per || b >= p.B) continue;
    const bool fits = at + gone[i] <= room;
    if (at <= room && !fits && rank == 0) report(p.err, PA_DEVERR_CAPACITY, b, gone[i]);
    s_at[b] = (int)min(at, 0x7fffffffll);
    s_from[b] = (keep[i] + ps - 1) >> p.page_log2;
    at += gone[i];
    if (fits) my_total = (int)at;
    else keep[i] = len[i];
  }
  __syncthreads();
  my_total = __reduce_max_sync(0xffffffffu, my_total);
  if ((tid & 31) == 0) atomicMax(&s_total, my_total);
  cluster.sync();  // the total; and every CTA has read the lengths and the count
  const int N = s_total;

  if (rank == 0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * per + i;
      if (i < per && b < p.B) p.seqlens_out[b] = keep[i];
    }
    if (tid == 0) *p.free_count_out = free_now + N;
  }
  const int lane = tid & 31;
  const Range r = warp_range(N, rank, ranks);
  auto give = [&](int b, int k, int page) {
    if (page < 0 || page >= p.num_pages) {
      report(p.err, PA_DEVERR_PAGE_OOB, b, s_from[b] + k - s_at[b]);
      s_bad = 1;
    }
    p.free_pages[free_now + k] = page;
  };
  auto entry_at = [&](int b) {  // the table entry of the request's released page 0, less its place
    return p.block_table + ((int64_t)b * p.bt_stride + s_from[b] - s_at[b]);
  };
  if (N >= 64 * p.B) {
    // Long runs: the warp copies one request's entries after another's, kAtOnce
    // of them in flight a lane.  Found one by one, below, they cost 100
    // instructions a line (179000 pages of 700 requests: 17.4 us, so 14.4 us),
    // but runs of a page or two would leave the lanes idle.
    for (int k0 = r.begin, b = 0; k0 < r.end;) {
      b = find_entry(s_at, p.B, b, k0);
      const int end = b + 1 < p.B ? min(r.end, s_at[b + 1]) : r.end;
      const int32_t* src = entry_at(b);
#pragma unroll 1
      for (int k = k0 + lane; k < end; k += 32 * kAtOnce) {
        int page[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) page[i] = load4(src + min(k + 32 * i, end - 1));
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          if (k + 32 * i < end) give(b, k + 32 * i, page[i]);
      }
      k0 = end;
    }
  } else {
    for (int k = r.begin + lane, b = 0; k < r.end; k += 32) {
      b = find_entry(s_at, p.B, b, k);
      give(b, k, load4(entry_at(b) + k));
    }
  }
  // A table entry outside the pool is not given back: CTA 0 closes the gaps.
  cluster.sync();  // the pages written, s_bad of every CTA
  int bad = 0;
  if (rank == 0)
    for (int r = 0; r < ranks; ++r) bad |= *cluster.map_shared_rank(&s_bad, r);
  cluster.sync();  // no CTA leaves while its s_bad is read
  if (rank != 0 || !bad) return;
  int32_t* list = p.free_pages + free_now;
  int kept = 0;
  for (int k0 = 0; k0 < N; k0 += (int)blockDim.x) {
    const int k = k0 + tid;
    const int page = k < N ? __ldcg(list + k) : -1;
    const bool ok = page >= 0 && page < p.num_pages;
    __syncthreads();  // the chunk read (and s_sums free) before anything is moved
    const int to = kept + (int)block_scan(ok ? 1 : 0, s_sums) - 1;
    if (ok) list[to] = page;
    __syncthreads();
    long long all = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) all += s_sums[w];
    kept += (int)all;
  }
  if (tid == 0) *p.free_count_out = free_now + kept;
}

// Whether the device schedules clusters of more than 8 CTAs of the kernel
// (sizes that are not portable); asked once a device.
template <typename K>
bool wide_clusters(K kernel, const cudaLaunchConfig_t& cfg, std::atomic<uint64_t>* asked,
                   std::atomic<uint64_t>* wide) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return false;
  const uint64_t bit = uint64_t(1) << dev;
  if ((asked->load(std::memory_order_acquire) & bit) == 0) {
    int n = 0;
    const bool ok =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
            cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0;
    if (!ok) cudaGetLastError();  // (not an error of the call's)
    if (ok) wide->fetch_or(bit, std::memory_order_relaxed);
    asked->fetch_or(bit, std::memory_order_release);
  }
  return (wide->load(std::memory_order_relaxed) & bit) != 0;
}

// `entry_bytes`: of shared memory for each entry of the batch.
template <typename P>
cudaError_t launch_cluster(void (*kernel)(P), const P& p, long long items, int entry_bytes,
                           cudaStream_t st) {
  // (one set a kernel: P tells them apart)
  static std::atomic<uint64_t> asked{0}, wide{0}, allowed{0};
  // For few entries and items one CTA of 256 threads, whose barriers are short;
  // otherwise as many CTAs as leave each thread two items.  16 CTAs instead of 8:
  // 1024 requests with 33000 new tokens 11.3 -> 8.9 us, 179000 pages of 700
  // finished requests 14.4 -> 11.5 us.
  const bool small = p.B <= 256 && items <= 512;
  int ctas = 1;
  while (ctas < kCluster && (long long)ctas * 2 * kThreads < items) ctas *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(small ? 256 : kThreads);
  cfg.dynamicSmemBytes = (size_t)p.B * entry_bytes;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)ctas;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cfg.dynamicSmemBytes > (40 << 10)) {  // with the static arrays more than the 48 KB of a plain launch
    // (the largest batch's: another thread's launch may be on its way)
    const cudaError_t e =
        allow_shared(reinterpret_cast<const void*>(kernel), kMaxB * entry_bytes, &allowed);
    if (e != cudaSuccess) return e;
  }
  if (ctas > 8 && !wide_clusters(kernel, cfg, &asked, &wide)) {
    cfg.gridDim = dim3(8);
    at.val.clusterDim.x = 8;
  }
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

int check_step(int B, int max_pages, int64_t bt_stride, int page_size, int64_t num_pages,
               int* page_log2) {
  if (B < 0) return set_error(PA_ERR_INVALID_ARG, "negative B");
  if (B > kMaxB) return set_error(PA_ERR_UNSUPPORTED, "more than %d sequences", kMaxB);
  if (max_pages < 1 || bt_stride < max_pages)
    return set_error(PA_ERR_INVALID_ARG,
                     "block table needs max_pages >= 1 and bt_stride >= max_pages");
  if (num_pages < 1 || num_pages > kMaxItems)
    return set_error(PA_ERR_INVALID_ARG, "num_pages must be in [1, 2^31 - 2^16]");
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) {
      *page_log2 = s;
      if (((long long)max_pages << s) > kMaxRowTokens)
        return set_error(PA_ERR_UNSUPPORTED,
                         "a block table row must hold at most 2^31 - 4096 tokens");
      return PA_OK;
    }
  return set_error(PA_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

PA_API int pa_plan_step(const int32_t* cache_seqlens, const int32_t* q_lens, int B,
                        int32_t* block_table, int64_t bt_stride, int max_pages, int page_size,
                        const int32_t* free_pages, const int32_t* free_count, int64_t num_pages,
                        int32_t* cu_seqlens_q, int32_t* seqlens_k, int64_t* slot_mapping,
                        int32_t* positions, int token_capacity, int32_t* free_count_out,
                        int32_t* err_word, pa_stream_t stream) {
  PlanParams p{};
  const int rc = check_step(B, max_pages, bt_stride, page_size, num_pages, &p.page_log2);
  if (rc) return rc;
  if (token_capacity < 0) return set_error(PA_ERR_INVALID_ARG, "negative token_capacity");
  if (token_capacity > kMaxItems)
    return set_error(PA_ERR_UNSUPPORTED, "token_capacity must be at most 2^31 - 2^16");
  if (cu_seqlens_q == nullptr || free_count == nullptr || free_count_out == nullptr ||
      free_pages == nullptr)
    return set_error(PA_ERR_INVALID_ARG,
                     "cu_seqlens_q, free_pages, free_count and free_count_out must be non-NULL");
  if (B > 0 && (cache_seqlens == nullptr || q_lens == nullptr || seqlens_k == nullptr ||
                block_table == nullptr))
    return set_error(PA_ERR_INVALID_ARG,
                     "cache_seqlens, q_lens, seqlens_k and block_table must be non-NULL");
  if (token_capacity > 0 && (slot_mapping == nullptr || positions == nullptr))
    return set_error(PA_ERR_INVALID_ARG, "slot_mapping and positions must be non-NULL");
  p.cache_seqlens = cache_seqlens;
  p.q_lens = q_lens;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.cu_seqlens_q = cu_seqlens_q;
  p.seqlens_k = seqlens_k;
  p.slots = slot_mapping;
  p.positions = positions;
  p.free_count_out = free_count_out;
  p.err = err_word;
  p.B = B;
  p.max_pages = max_pages;
  p.token_capacity = token_capacity;
  p.num_pages = (int)num_pages;
  const cudaError_t e = launch_cluster(plan_kernel, p, token_capacity,
                                       3 * (int)sizeof(int),
                                       reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(PA_ERR_CUDA, "plan launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

PA_API int pa_release_pages(const int32_t* cache_seqlens, const int32_t* keep_lens, int B,
                            const int32_t* block_table, int64_t bt_stride, int max_pages,
                            int page_size, int32_t* free_pages, const int32_t* free_count,
                            int64_t num_pages, int32_t* seqlens_out, int32_t* free_count_out,
                            int32_t* err_word, pa_stream_t stream) {
  ReleaseParams p{};
  const int rc = check_step(B, max_pages, bt_stride, page_size, num_pages, &p.page_log2);
  if (rc) return rc;
  if (free_count == nullptr || free_count_out == nullptr || free_pages == nullptr)
    return set_error(PA_ERR_INVALID_ARG,
                     "free_pages, free_count and free_count_out must be non-NULL");
  if (B > 0 && (cache_seqlens == nullptr || keep_lens == nullptr || seqlens_out == nullptr ||
                block_table == nullptr))
    return set_error(PA_ERR_INVALID_ARG,
                     "cache_seqlens, keep_lens, seqlens_out and block_table must be non-NULL");
  p.cache_seqlens = cache_seqlens;
  p.keep_lens = keep_lens;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.seqlens_out = seqlens_out;
  p.free_count_out = free_count_out;
  p.err = err_word;
  p.B = B;
  p.max_pages = max_pages;
  p.num_pages = (int)num_pages;
  const long long most = (long long)B * max_pages;
  const cudaError_t e = launch_cluster(release_kernel, p, most < num_pages ? most : num_pages,
                                       2 * (int)sizeof(int),
                                       reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(PA_ERR_CUDA, "release launch: %s", cudaGetErrorString(e));
  return PA_OK;
}

}  // extern "C"
