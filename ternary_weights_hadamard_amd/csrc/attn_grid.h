// How many workgroups a tb_paged_attention call has work for, from what the
// host knows, and which head a workgroup's work is of.  Plain C++, so that it is
// also tested on the host.
#pragma once

#include "paged.h"

namespace tb {

// A launch's x extent: with 256 threads each below the 2^32 threads that it may
// have.  More workgroups go on in y (of at most 2^36 + 2^33, as tb.h bounds them).
constexpr int64_t kMaxGridX = (int64_t)1 << 23;

struct GridXY {
  unsigned x, y;
};
inline GridXY grid_of(int64_t blocks) {
  const int64_t x = blocks < kMaxGridX ? blocks : kMaxGridX;
  return GridXY{(unsigned)x, (unsigned)((blocks + x - 1) / x)};
}

// Most tokens of a sequence that are computed: max_q may be far above every length.
inline int64_t most_tokens(int64_t max_q, int64_t total_q) { return max_q < total_q ? max_q : total_q; }

// Row tiles of `tile` rows, at most, that the sequences of more than `few` rows
// have for one key/value head: only so many sequences have as many tokens, and
// each has less than one tile more than its share of all rows.
inline int64_t most_row_tiles(int64_t total_q, int64_t B, int64_t group, int64_t few, int64_t tile) {
  const int64_t some = total_q / (few / group + 1);
  return total_q * group / tile + (B < some ? B : some);
}

// The head whose `tiles` hold place `at`, all heads' in order: heads * tiles pass
// 32 bits (129 heads of 2^30 positions), but 64-bit divisions are long.
TB_HOST_DEVICE int head_of(int64_t at, int tiles) {
  return at >> 32 == 0 ? (int)((uint32_t)at / (uint32_t)tiles) : (int)(at / tiles);
}

}  // namespace tb
