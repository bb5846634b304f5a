// The plan of a tb_paged_attention call and the output of a row.
#pragma once

#include "attn_common.h"

namespace tb {

// A sequence with few rows (attn_line.h) goes to the kernel for those, the
// others to the chunk kernel.  Parts in the workspace, for each kind:
//   values  float  [2 pieces][rows of a row tile][D]  (not divided by the sum)
//   stats   float2 [2 pieces][rows of a row tile]     (what both are relative to, in log2 units; sum)
struct AttnLine {
  int pieces;     // workgroups; 0: one for each item, none is in parts
  int least;      // tiles of a piece
  int slot_rows;  // rows of a slot
  float* values;
  float2* stats;
  // tiles of a piece of a line of `total`
  __host__ __device__ int64_t piece(int64_t total) const {
    const int64_t sum = total + pieces - 1;
    const int64_t per = sum >> 32 == 0 ? (int64_t)((uint32_t)sum / (uint32_t)pieces) : sum / pieces;
    return per < least ? least : per;
  }
};

struct AttnPlan {
  int64_t few;       // most rows of the first kind (0: all sequences are of the second)
  int64_t capacity;  // positions that the table has room for
  int group;         // query heads of a key/value head
  int shift;         // log2 of a page's positions
  int64_t chunk_blocks;  // workgroups of chunks: they come first
  AttnLine rows_line, chunk_line;
  __host__ __device__ bool is_chunk(int64_t nrows) const { return nrows > few; }
};

constexpr int kAttnWaves = 4;    // waves of a workgroup
constexpr int kRowsTile = 16;    // rows of a row tile: few rows,
constexpr int kChunkTile = 128;  // and chunks
// positions of a tile: few rows (the cache's type), and chunks
__host__ __device__ constexpr int rows_positions(bool fp8) { return fp8 ? 64 : 32; }
constexpr int kChunkPositions = 64;

// The tiles that hold a span's positions: first .. first + count - 1.
struct TileSpan {
  int first, count;
};
__device__ __forceinline__ TileSpan tile_span(const PagedSpan& p, int positions) {
  const int first = p.begin / positions;
  return TileSpan{first, p.end > p.begin ? (p.end + positions - 1) / positions - first : 0};
}

// A workgroup's LDS.  Few rows: a buffer and 16 of max and of sum for each
// wave.  Chunks: K of two tiles, V of two tiles.
struct AttnShared {
  u32x4* buffer[4];
  float *max, *sum;
  int* bits;        // of each wave, for what all waves have to know
  uint32_t* marks;  // of chunks: values that are not finite (attn_chunk.h)
};

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
