// Where a sequence's tokens and positions lie in the paged cache, and what of
// it exists.  Everything that reaches memory through cu_q, kv_len or
// block_table goes through these functions; they are plain C++, so that they
// are also tested on the host with entries that are wrong.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>
#define TB_HOST_DEVICE __host__ __device__ inline
#else
#define TB_HOST_DEVICE inline
#endif

namespace tb {

struct PagedSeq {
  int64_t row0;   // first row of the token arrays
  int n;          // new tokens
  int keys;       // positions 0 .. keys - 1 may exist (inside the table)
  int first_pos;  // position of token 0 (negative: it has none)
};

// Sequence b: rows clamped to [0, total_q], positions to the table.
TB_HOST_DEVICE PagedSeq paged_seq(const int32_t* cu_q, const int32_t* kv_len, int64_t b, int64_t total_q,
                                  int64_t capacity) {
  PagedSeq s;
  int64_t lo = cu_q[b], hi = cu_q[b + 1];
  lo = lo < 0 ? 0 : lo > total_q ? total_q : lo;
  hi = hi < lo ? lo : hi > total_q ? total_q : hi;
  const int kv = kv_len[b] < 0 ? 0 : kv_len[b];
  s.row0 = lo;
  s.n = (int)(hi - lo);
  s.keys = kv < capacity ? kv : (int)capacity;
  s.first_pos = kv - s.n;
  return s;
}

// The page of entry `i` of a sequence's table row, or -1 if there is none; in
// two steps where the entry is used long after it was asked for.
TB_HOST_DEVICE int32_t paged_entry(const int32_t* row, int64_t width, int64_t i) {
  int32_t id = -1;
  if (i >= 0 && i < width) id = row[i];
  return id;
}
TB_HOST_DEVICE int paged_id(int32_t entry, int64_t n_pages) { return entry >= 0 && entry < n_pages ? entry : -1; }
TB_HOST_DEVICE int paged_page(const int32_t* row, int64_t width, int64_t n_pages, int64_t i) {
  return paged_id(paged_entry(row, width, i), n_pages);
}

// What an e4m3 code of a head is multiplied with.
TB_HOST_DEVICE float head_scale(const void* scales, int head) {
  return scales ? static_cast<const float*>(scales)[head] : 1.f;
}

// The positions that some of the tokens j0 .. j1 (inclusive, j1 < n) see: [begin, end).
struct PagedSpan {
  int begin, end;
};
TB_HOST_DEVICE PagedSpan paged_span(const PagedSeq& s, int j0, int j1, int64_t window) {
  PagedSpan r;
  const int64_t top = (int64_t)s.first_pos + j1 + 1;  // the last token's position + 1
  int64_t low = window > 0 ? (int64_t)s.first_pos + j0 - window + 1 : 0;
  if (low < 0) low = 0;
  r.end = top < 0 ? 0 : top < s.keys ? (int)top : s.keys;
  r.begin = low < r.end ? (int)low : r.end;
  return r;
}

}  // namespace tb
