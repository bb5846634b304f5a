// The plan of a tb_paged_attention call and the output of a row.
#pragma once

#include "attn_common.h"

namespace tb {

// Rows are the (token, head) pairs of one key/value head of one sequence.  A
// sequence with few of them goes to the kernel for few rows, the others to
// the chunk kernel; a launch's workgroups for sequences that are not its own
// end at once.
//
// Chunks: the positions that a row tile sees are cut into parts of a fixed
// length (the last part of a launch's `splits` takes what is left).  Few rows:
// all tiles of all items stand in one line that is cut into equal pieces, each
// with the parts of at most two items.  An item in one part is written by its
// kernel, the others are joined from the workspace:
//   values, stats            [part][row]: of chunks, row of total_q * heads_q
//   rows_values, rows_stats  [2 pieces + 0 or 1][row of the item]
// with D floats (not divided by the sum) and a float2 (maximum in log2 units,
// sum) a row.  A chunk's part with a sum of 0 has no values.
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
  int64_t few;       // most rows of the first kind
  int64_t rows;      // total_q * heads_q
  int64_t capacity;  // positions that the table has room for
  int group;         // query heads of a key/value head
  int shift;         // log2 of a page's positions
  int pieces;        // workgroups of the first kind; 0: one for each item, in one part
  int least;         // tiles of a piece
  int slot_rows;     // rows of a slot of the workspace
  unsigned chunk_blocks;  // workgroups of the second kind for each sequence
  AttnSplit by_chunk;
  float *values, *rows_values;
  float2 *stats, *rows_stats;
  __host__ __device__ bool is_chunk(int64_t nrows) const { return nrows > few; }
  // tiles of a piece of a line of `total`
  __host__ __device__ int64_t piece(int64_t total) const {
    const int64_t per = (total + pieces - 1) / pieces;
    return per < least ? least : per;
  }
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
