// Shared by the two kernels of pa_fwd_varlen_e4m3: parameters, the sequences
// of a ragged batch, and the conversion of e4m3 values.
#pragma once

#include <cuda_fp8.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

constexpr float kE4m3Shift = 10.f;  // log2 of what probabilities are scaled by
constexpr float kE4m3Slack = 5.f;   // log2 of how far they may pass that

struct AttendParams {
  const void* q;
  int64_t q_st, q_sh;
  const uint8_t *k_cache, *v_cache;
  int64_t k_sb, k_st, k_sh, v_sb, v_st, v_sh;
  const float *k_scale, *v_scale;
  const int32_t *cu_seqlens_q, *seqlens_k, *block_table;
  int64_t bt_stride, num_pages;
  int B, total_q, Hq, Hkv, G, max_pages, page_shift, max_seqlen_k, causal;
  int small_rows;  // sequences of at most this many rows per kv head run on the warp-level kernel
  float scale_log2;
  void* out;
  float* lse;
  // Split results: two a CTA, one of the stream that began before its share
  // and one of the stream that goes on behind it.
  unsigned long long* words;  // [CTAs] arrivals on the stream that starts in the CTA and goes on
  float2* part_ml;            // reference and sum of each row
  float* part_o;
  int32_t* err;
};

// a / b of non-negative values, in 32 bits where they do.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

struct SeqRows {
  int q0, qlen, lk;
};

// The rows and keys of sequence b: offsets kept within the packed rows, a
// length that the table or max_seqlen_k does not hold run as 0.
__device__ __forceinline__ SeqRows seq_rows(const AttendParams& p, int b, bool tell) {
  SeqRows s{};
  const int c0 = __ldg(p.cu_seqlens_q + b), c1 = __ldg(p.cu_seqlens_q + b + 1);
  s.q0 = min(max(c0, 0), p.total_q);
  s.qlen = min(max(c1, s.q0), p.total_q) - s.q0;
  s.lk = __ldg(p.seqlens_k + b);  // (not behind the offsets: one latency, not two)
  if (s.qlen == 0) {
    s.lk = 0;
    return s;
  }
  const long long cap = (long long)p.max_pages * (kPage << p.page_shift);
  if (s.lk < 0 || s.lk > p.max_seqlen_k || s.lk > cap) {
    if (tell) report(p.err, PA_DEVERR_LENGTH, b, s.lk);
    s.lk = 0;
  }
  return s;
}

// Two e4m3 values (the low byte first) as two fp16 values.
__device__ __forceinline__ uint32_t f16x2_of(uint32_t e4m3x2) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)e4m3x2));
  return h;
}
// Four e4m3 values (the low byte first) as two pairs of fp16 values.
__device__ __forceinline__ void f16x4_of(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float x;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(x) : "f"(a), "f"(b), "f"(c));
  return x;
}
// The sign bits (moved to bit 7) of the NaN bytes among four e4m3 values.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// The attention of sequences of more than small_rows rows per kv head
// (chunk_e4m3.cu).
cudaError_t launch_chunks_e4m3(const AttendParams& p, int D, int dtype, cudaStream_t st);
constexpr int kChunkRows = 256;  // rows of its pair of query tiles: part_ml [2 CTAs][256],
                                 // part_o [2 CTAs][2 tiles][D / 4][128][4]

}  // namespace pa
