// How the work of a tb_paged_attention call is cut.
//
// Rows are the (token, head) pairs of one key/value head of one sequence, in
// tiles; positions are in tiles too.  An item is one row tile of one key/value
// head of one sequence: it reads the position tiles that some of its rows see.
// The tiles of all items of a kind stand in one line, ordered by sequence, row
// tile and head, and the line is cut into equal pieces, one for each workgroup
// that the GPU holds, so that batches of mixed lengths end everywhere at once.
// A piece covers some items whole, which it writes, and parts of at most two,
// which go to the workspace and are joined by a second launch.  Nothing is
// read back to the host: every workgroup finds its piece from cu_q and kv_len.
#pragma once

#include "attn_grid.h"
#include "attn_launch.h"
#include "wave_scan.h"

namespace tb {

// a value that is the same in every lane, in scalar registers
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = (uint32_t)uniform((int)(uint32_t)v), hi = (uint32_t)uniform((int)(uint32_t)((uint64_t)v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// A sequence as one kind sees it.
struct LineSeq {
  PagedSeq seq;
  int rows;  // 0: it is of the other kind
};

template <bool CHUNK, bool FP8>
struct LineKind {
  static constexpr int kRows = CHUNK ? kChunkTile : kRowsTile;
  static constexpr int kPositions = CHUNK ? kChunkPositions : rows_positions(FP8);

  static __device__ __forceinline__ LineSeq sequence(const tb_paged_attention_args& a, const AttnPlan& plan, int64_t b) {
    const tb_paged_cache& c = a.cache;
    LineSeq s;
    s.seq = paged_seq(c.cu_q, c.kv_len, b, c.total_q, plan.capacity);
    const int rows = (s.seq.n < (int)c.max_q ? s.seq.n : (int)c.max_q) * plan.group;
    s.rows = plan.is_chunk(rows) == CHUNK ? rows : 0;
    return s;
  }
  static __device__ __forceinline__ PagedSpan span(const tb_paged_attention_args& a, const AttnPlan& plan,
                                                   const LineSeq& s, int rt) {
    const int r0 = rt * kRows, rl = r0 + kRows - 1 < s.rows ? r0 + kRows - 1 : s.rows - 1;
    return paged_span(s.seq, (unsigned)r0 / (unsigned)plan.group, (unsigned)rl / (unsigned)plan.group, a.window);
  }
  // Tiles of the row tile's items in the line: those that hold a position it
  // sees, or one (empty) in which its rows are written.
  static __device__ __forceinline__ int tiles(const tb_paged_attention_args& a, const AttnPlan& plan, const LineSeq& s,
                                              int rt) {
    const int n = tile_span(span(a, plan, s, rt), kPositions).count;
    return n > 1 ? n : 1;
  }
  // of row tiles 0 .. count - 1, for one head; a whole wave, the same arguments in every lane
  static __device__ __forceinline__ int64_t tiles_before(const tb_paged_attention_args& a, const AttnPlan& plan,
                                                         const LineSeq& s, int count) {
    int64_t n = 0;
    for (int rt = threadIdx.x & 63; rt < count; rt += 64) n += tiles(a, plan, s, rt);
    return wave_sum(n);
  }
};

__device__ __forceinline__ LineSeq uniform_seq(const LineSeq& x, int lane) {
  LineSeq r;
  r.seq.row0 = of_lane(x.seq.row0, lane);
  r.seq.n = __builtin_amdgcn_readlane(x.seq.n, lane);
  r.seq.keys = __builtin_amdgcn_readlane(x.seq.keys, lane);
  r.seq.first_pos = __builtin_amdgcn_readlane(x.seq.first_pos, lane);
  r.rows = __builtin_amdgcn_readlane(x.rows, lane);
  return r;
}

struct LineItem {
  int64_t start;  // of its first tile in the line
  int tiles;      // in the line
  int64_t b;
  int rt, head;
  LineSeq seq;
  PagedSpan span;
  TileSpan held;  // the tiles that hold a position some row sees
};

// an item, the same in every lane, in scalar registers
__device__ __forceinline__ LineItem uniform_item(const LineItem& x) {
  LineItem r;
  r.start = uniform64(x.start);
  r.tiles = uniform(x.tiles);
  r.b = uniform64(x.b);
  r.rt = uniform(x.rt);
  r.head = uniform(x.head);
  r.seq = uniform_seq(x.seq, 0);
  r.span.begin = uniform(x.span.begin);
  r.span.end = uniform(x.span.end);
  r.held.first = uniform(x.held.first);
  r.held.count = uniform(x.held.count);
  return r;
}

// The line of one kind.  Whole waves use it together, with the same arguments
// in every lane, and all lanes active: the lanes take a sequence each, and for
// one of many row tiles a row tile each.
template <bool CHUNK, bool FP8>
struct Line {
  typedef LineKind<CHUNK, FP8> K;
  LineSeq own;    // of sequence b0 + lane, of the last 64 looked at
  int64_t up;     // tiles of the sequences b0 .. b0 + lane
  int64_t total;  // tiles of the line

  __device__ __forceinline__ void look(const tb_paged_attention_args& a, const AttnPlan& plan, int64_t b0) {
    const int lane = threadIdx.x & 63;
    own = LineSeq{};
    int64_t n = 0;
    if (b0 + lane < a.cache.B) {
      own = K::sequence(a, plan, b0 + lane);
      if (own.rows > 0) n = K::tiles(a, plan, own, 0);
    }
    if constexpr (CHUNK) {
      for (uint64_t more = __ballot(own.rows > K::kRows); more != 0; more &= more - 1) {
        const int l = uniform(__builtin_ctzll(more));
        const LineSeq s = uniform_seq(own, l);
        const int64_t t = K::tiles_before(a, plan, s, (s.rows + K::kRows - 1) / K::kRows);
        if (lane == l) n = t;
      }
    }
    up = wave_prefix(n * a.cache.heads_kv);
  }
  __device__ __forceinline__ Line(const tb_paged_attention_args& a, const AttnPlan& plan) {
    total = 0;
    for (int64_t b0 = 0; b0 < a.cache.B; b0 += 64) {
      look(a, plan, b0);
      total += of_lane(up, 63);
    }
  }
  // The item that holds tile `at` < total.
  __device__ __forceinline__ LineItem find(const tb_paged_attention_args& a, const AttnPlan& plan, int64_t at) {
    LineItem it{};
    int64_t before = 0;
    for (int64_t b0 = 0; b0 < a.cache.B; b0 += 64) {
      if (a.cache.B > 64) look(a, plan, b0);  // else it holds them since it was made
      const uint64_t past = __ballot(before + up > at);
      if (past != 0) {
        const int l = uniform(__builtin_ctzll(past));
        it.b = b0 + l;
        it.start = before + (l > 0 ? of_lane(up, l - 1) : 0);
        it.seq = uniform_seq(own, l);
        break;
      }
      before += of_lane(up, 63);
    }
    const int64_t heads = a.cache.heads_kv;
    if constexpr (CHUNK) {
      for (int rt0 = 0; rt0 * K::kRows < it.seq.rows; rt0 += 64) {
        const int rt = rt0 + (threadIdx.x & 63);
        const int64_t n = rt * K::kRows < it.seq.rows ? heads * K::tiles(a, plan, it.seq, rt) : 0, ends = wave_prefix(n);
        const uint64_t past = __ballot(it.start + ends > at);
        if (past != 0) {
          const int l = uniform(__builtin_ctzll(past));
          it.rt = rt0 + l;
          it.start += of_lane(ends, l) - of_lane(n, l);
          break;
        }
        it.start += of_lane(ends, 63);
      }
    }
    set(a, plan, it);
    it.head = head_of(at - it.start, it.tiles);
    it.start += (int64_t)it.head * it.tiles;
    return uniform_item(it);
  }
  // what follows from an item's sequence and row tile
  static __device__ __forceinline__ void set(const tb_paged_attention_args& a, const AttnPlan& plan, LineItem& it) {
    it.span = K::span(a, plan, it.seq, it.rt);
    it.held = tile_span(it.span, K::kPositions);
    it.tiles = it.held.count > 1 ? it.held.count : 1;
  }
  // The item behind `it`, which is not the line's last.
  static __device__ __forceinline__ LineItem next(const tb_paged_attention_args& a, const AttnPlan& plan, LineItem it) {
    it.start += it.tiles;
    if (++it.head < a.cache.heads_kv) return it;
    it.head = 0;
    if (CHUNK && ++it.rt * K::kRows < it.seq.rows) {
      set(a, plan, it);
      return uniform_item(it);
    }
    it.rt = 0;
    for (++it.b; it.b < a.cache.B; it.b += 64) {
      LineSeq own{};
      if (it.b + (threadIdx.x & 63) < a.cache.B) own = K::sequence(a, plan, it.b + (threadIdx.x & 63));
      const uint64_t some = __ballot(own.rows > 0);
      if (some != 0) {
        const int l = uniform(__builtin_ctzll(some));
        it.b += l;
        it.seq = uniform_seq(own, l);
        break;
      }
    }
    set(a, plan, it);
    return uniform_item(it);
  }
  // Where the items of sequence b start.
  __device__ __forceinline__ int64_t before(const tb_paged_attention_args& a, const AttnPlan& plan, int64_t b) {
    int64_t n = 0;
    for (int64_t b0 = 0; b0 <= b; b0 += 64) {
      if (a.cache.B > 64) look(a, plan, b0);
      if (b - b0 < 64) return n + (b > b0 ? of_lane(up, (int)(b - b0) - 1) : 0);
      n += of_lane(up, 63);
    }
    return n;
  }
};

// The parts of the item whose tiles stand at start .. start + tiles - 1 of a
// line of pieces of `per` tiles.
struct LineParts {
  int64_t first;  // piece
  int count;
  int64_t slot0;  // of the first part; part p > 0 has slot 2 (first + p)
  __device__ __forceinline__ int64_t slot(int p) const { return p == 0 ? slot0 : 2 * (first + p); }
};
__device__ __forceinline__ LineParts line_parts(int64_t start, int tiles, int64_t per) {
  LineParts r;
  const int64_t last = start + tiles - 1;
  if (last >> 32 == 0 && per >> 32 == 0) {  // 64-bit divisions are long
    r.first = (uint32_t)start / (uint32_t)per;
    r.count = (int)((uint32_t)last / (uint32_t)per - (uint32_t)r.first) + 1;
  } else {
    r.first = start / per;
    r.count = (int)(last / per - r.first) + 1;
  }
  // a piece's first part has slot 2 piece, the part it ends with slot 2 piece + 1
  r.slot0 = 2 * r.first + (r.first * per < start ? 1 : 0);
  return r;
}

// Item `at` of a line that is not cut; false if there is none.  Chunks: of the
// items that exist, so that how far max_q is above the lengths costs nothing;
// the last rows of a sequence see the most positions and go first.  Few rows: a
// sequence has one for each head, and none if it is of the other kind.  Whole
// waves, the same arguments in every lane.
template <bool CHUNK, bool FP8>
__device__ __forceinline__ bool uncut_item(const tb_paged_attention_args& a, const AttnPlan& plan, int64_t at,
                                           LineItem& it) {
  typedef LineKind<CHUNK, FP8> K;
  const int64_t heads = a.cache.heads_kv;
  it = LineItem{};
  int64_t t = at >> 32 == 0 ? (int64_t)((uint32_t)at / (uint32_t)heads) : at / heads;
  it.head = (int)(at - t * heads);
  if constexpr (CHUNK) {
    constexpr int kAhead = 4;  // of 64 sequences, whose lengths are loaded together
    const int lane = threadIdx.x & 63;
    for (int64_t b0 = 0; it.seq.rows == 0; b0 += 64 * kAhead) {
      if (b0 >= a.cache.B) return false;
      LineSeq own[kAhead];
      int64_t n[kAhead], sum = 0;  // row tiles
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t b = b0 + 64 * u + lane;
        own[u] = LineSeq{};
        if (b < a.cache.B) own[u] = K::sequence(a, plan, b);
        n[u] = (own[u].rows + K::kRows - 1) / K::kRows;
        sum += n[u];
      }
      sum = wave_sum(sum);
      if (t >= sum) {
        t -= sum;
        continue;
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (it.seq.rows != 0) continue;
        const int64_t up = wave_prefix(n[u]);
        const uint64_t past = __ballot(up > t);
        if (past == 0) {
          t -= of_lane(up, 63);
          continue;
        }
        const int l = uniform(__builtin_ctzll(past));
        it.b = b0 + 64 * u + l;
        it.rt = (int)(of_lane(up, l) - 1 - t);
        it.seq = uniform_seq(own[u], l);
      }
    }
  } else {
    if (t >= a.cache.B) return false;
    it.b = t;
    it.seq = K::sequence(a, plan, t);
    if (it.seq.rows == 0) return false;
  }
  Line<CHUNK, FP8>::set(a, plan, it);
  it = uniform_item(it);
  return true;
}

// What workgroup `block` does: all parts of its piece of the line, or, if the
// line is not cut, its item.  part(item, t0, t1, slot, careful) does tiles t0 ..
// t1 - 1 of an item, all of them if slot < 0; if it answers true it is to be done
// again, carefully.  LDS is free for it when it is called, and when it answers.
template <bool CHUNK, bool FP8, typename F>
__device__ __forceinline__ void run_line(const tb_paged_attention_args& a, const AttnPlan& plan, int64_t block, F part) {
  const AttnLine& cut = CHUNK ? plan.chunk_line : plan.rows_line;
  bool careful = false;
  LineItem it;
  int64_t at, end;
  if (cut.pieces == 0) {
    if (!uncut_item<CHUNK, FP8>(a, plan, block, it)) return;
    if constexpr (CHUNK) {
      // a copy of its own: with what the loop over a piece's parts holds, the
      // chunk kernel runs out of scalar registers (4 x 2048 tokens 5 % slower)
      do {
        careful = uniform(part(it, 0, it.tiles, (int64_t)-1, careful));
      } while (careful);
      return;
    }
    at = it.start = 0;
    end = it.tiles;
  } else {
    Line<CHUNK, FP8> line(a, plan);
    const int64_t per = cut.piece(line.total);
    at = uniform64(block * per);
    end = uniform64(at + per < line.total ? at + per : line.total);
    if (at >= end) return;
    it = line.find(a, plan, at);
  }
  for (int nth = 0;;) {
    const int t0 = uniform((int)(at - it.start));
    const int t1 = uniform(it.start + it.tiles < end ? it.tiles : (int)(end - it.start));
    careful = uniform(part(it, t0, t1, t0 == 0 && t1 == it.tiles ? (int64_t)-1 : 2 * block + nth, careful));
    if (careful) continue;
    nth = 1;
    at = it.start + t1;
    if (at >= end) return;
    __syncthreads();  // the next part writes the LDS that this one reads
    it = Line<CHUNK, FP8>::next(a, plan, it);
  }
}

}  // namespace tb
