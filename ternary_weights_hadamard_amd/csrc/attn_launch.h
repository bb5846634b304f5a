// The plan of a tb_paged_attention call, the kernels it launches, and the
// output of a row.
#pragma once

#include "attn_common.h"

namespace tb {

// Rows are the (token, head) pairs of one key/value head of one sequence.  A
// sequence with few of them goes to the kernel for few rows, the others to
// the chunk kernel; a launch's workgroups for sequences that are not its own
// end at once.  Each kind's positions are split over its own number of parts.
// A part's statistics and weighted values in the workspace, parts of all rows
// after one another:
//   values  float  [parts][rows][D]  (not divided by the sum)
//   stats   float2 [parts][rows]     (maximum in log2 units, sum; no values are
//                                     written or read where the sum is 0)
struct AttnPlan {
  int64_t few;  // most rows of the first kind
  int64_t rows; // total_q * heads_q
  int rows_splits, chunk_splits;
  float* values;
  float2* stats;
  __host__ __device__ bool by_chunk(int64_t nrows) const { return nrows > few; }
};

hipError_t launch_attn_rows(const tb_paged_attention_args& a, const AttnPlan& plan, hipStream_t stream);
hipError_t launch_attn_chunk(const tb_paged_attention_args& a, const AttnPlan& plan, hipStream_t stream);

// What a row's weighted values are multiplied with; its log-sum-exp is
// written on the way (`first`: by the one lane that does).
struct RowScale {
  float f;
};
__device__ __forceinline__ RowScale row_scale(const tb_paged_attention_args& a, int head, int64_t at, bool first,
                                              float top, float total) {
  const tb_paged_cache& c = a.cache;
  const float vs = c.cache_dtype == TB_FP8 && c.v_scale ? c.v_scale[head] : 1.f;
  if (a.lse && first) a.lse[at] = total == 0.f ? -__builtin_inff() : (top + log2f(total)) * kLn2;
  return RowScale{total == 0.f ? 0.f : vs / total};
}

// Four channels of the output from element `i` on.
__device__ __forceinline__ void write4(const tb_paged_attention_args& a, int64_t i, const f32x4& v, const RowScale& s) {
  const f32x4 w = v * s.f;
  if (a.out_dtype == TB_F32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + i) = w;
  } else {
    u32x2 h;
    h[0] = f32_to_bf16_rne(w[0]) | (f32_to_bf16_rne(w[1]) << 16);
    h[1] = f32_to_bf16_rne(w[2]) | (f32_to_bf16_rne(w[3]) << 16);
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + i) = h;
  }
}

}  // namespace tb
