// The plan of a tb_paged_attention call, the kernels it launches, and the
// output of a row.
#pragma once

#include "attn_common.h"

namespace tb {

// Rows are the (token, head) pairs of one key/value head of one sequence.  A
// sequence with few of them goes to the kernel for few rows, the others to
// the chunk kernel; a launch's workgroups for sequences that are not its own
// end at once.
//
// The positions that a workgroup's rows see are cut into parts of a fixed
// length, so that sequences of different lengths give equal pieces of work;
// only the last part of a launch's `splits` takes what is left.  A row tile
// with one part is written by its kernel, the others are joined from the
// workspace, where the parts of all rows lie after one another:
//   values  float  [parts][rows][D]  (not divided by the sum)
//   stats   float2 [parts][rows]     (maximum in log2 units, sum; no values are
//                                     written or read where the sum is 0)
struct AttnSplit {
  int splits;  // most parts (the grid's)
  int tiles;   // tiles of a part
  // parts that a row tile with this many tiles of positions is cut into
  __host__ __device__ int parts(int all) const {
    const int p = (all + tiles - 1) / tiles;
    return p < 1 ? 1 : p > splits ? splits : p;
  }
};

struct AttnPlan {
  int64_t few;   // most rows of the first kind
  int64_t rows;  // total_q * heads_q
  AttnSplit by_rows, by_chunk;
  float* values;
  float2* stats;
  __host__ __device__ bool is_chunk(int64_t nrows) const { return nrows > few; }
};

constexpr int kRowsTile = 16;    // rows of a workgroup: few rows,
constexpr int kChunkTile = 128;  // and chunks
// positions of a tile: few rows (the cache's type), and chunks
__host__ __device__ constexpr int rows_positions(bool fp8) { return fp8 ? 64 : 32; }
constexpr int kChunkPositions = 64;

// The tiles of positions that the rows r0 .. r0 + rows - 1 see: [first, first + count).
struct TileSpan {
  int first, count;
};
__device__ __forceinline__ TileSpan tile_span(const PagedSpan& p, int positions) {
  const int first = p.begin / positions;
  return TileSpan{first, p.end > p.begin ? (p.end + positions - 1) / positions - first : 0};
}

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
