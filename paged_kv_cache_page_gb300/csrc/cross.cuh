// Attention of a ragged batch's rows to the keys of their entry (pa_fwd_cross):
// what its two kernels share.
#pragma once

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

struct CrossParams {
  const void* q;
  int64_t q_st, q_sh;
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* lens_k;    // or null
  const uint8_t* key_mask;  // or null
  int B, total_q, total_k, max_q, max_k, Hq, Hkv, G;
  float scale_log2;
  void* out;
  float* lse;
  int32_t* err;
  // The wide kernel takes at most 128 heads at a time: a kv head with more counts as
  // kv_split of them (Hkv and G above are then those).  Its parts of cut streams:
  int kv_split;
  unsigned long long* words;
  float2* part_ml;
  float* part_o;
};

// A load that stays where it is written (see load16).
__device__ __forceinline__ uint32_t load_byte(const uint8_t* src) {
  uint32_t x;
  asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(x) : "l"(src));
  return x;
}

// Rows [q0, q0 + rows) of q and keys [k0, k0 + keys) of k and v.
struct CrossEntry {
  int q0, rows, k0, keys;
};
__device__ __forceinline__ CrossEntry cross_entry(const CrossParams& p, int b, bool rep) {
  CrossEntry e;
  e.q0 = __ldg(p.cu_q + b);
  const long long rows = (long long)__ldg(p.cu_q + b + 1) - e.q0;
  e.k0 = __ldg(p.cu_k + b);
  const long long room = (long long)__ldg(p.cu_k + b + 1) - e.k0;
  const long long keys = p.lens_k != nullptr ? __ldg(p.lens_k + b) : room;
  const bool rows_ok =
      e.q0 >= 0 && rows >= 0 && e.q0 + rows <= p.total_q && rows <= p.max_q;
  const bool keys_ok = e.k0 >= 0 && keys >= 0 && keys <= room && e.k0 + keys <= p.total_k &&
                       keys <= p.max_k;
  if (rep && !(rows_ok && keys_ok))
    report(p.err, PA_DEVERR_LENGTH, b, (int)(rows_ok ? keys : rows));
  // (rows that lie in q are written; they have no keys where a length is malformed)
  const long long most = min((long long)p.total_q - max(e.q0, 0), (long long)p.max_q);
  e.rows = e.q0 < 0 ? 0 : (int)max(0ll, min(rows, most));
  e.keys = rows_ok && keys_ok ? (int)keys : 0;
  return e;
}

// Few rows: warp-level MMAs, clusters over the keys.  Many rows: tcgen05.
cudaError_t launch_cross_narrow(const CrossParams& p, const CUtensorMap& tmk,
                                const CUtensorMap& tmv, int D, int dtype, cudaStream_t st);
// tmq: q with boxes of 64 columns, G heads, 128 / G rows; tmk, tmv: 64 columns, 128 keys.
cudaError_t launch_cross_wide(CrossParams p, const CUtensorMap& tmq, const CUtensorMap& tmk,
                              const CUtensorMap& tmv, int D, int dtype, void* workspace,
                              cudaStream_t st);
size_t cross_wide_workspace(int D);
constexpr int cross_narrow_box(int D) { return D == 64 ? 32 : 16; }  // keys of a box

}  // namespace pa
