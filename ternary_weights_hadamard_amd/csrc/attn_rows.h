// Attention over the paged cache for few rows: a decode step's token, or a
// handful of drafted ones, of every head that shares a key/value head
// (include/tb.h, tb_paged_attention).
//
// Mathematics.  Rows (token, head) of one key/value head are the 16 columns of
// S' = K Q' (v_mfma 16x16x32), so a lane holds the scores of one row for
// positions that are its own, and their weights are, without any exchange,
// the operand of O' = V' P': the positions that matrix row m of K stands for
// are chosen so that a lane's eight weights of a 32-position block belong to
// eight consecutive positions, which is one 16-byte load of a V page
// ([d][position]) for bf16; for e4m3 two blocks share a load of 16 positions.
// The running maximum and sum of each row are kept in log2 units.
//
// What bounds it: the cache's bytes.  Every K and V byte is loaded once,
// straight into operand registers (no LDS, no barrier in the loop), and two
// tiles of a wave are in flight: each half of a tile's registers is loaded
// again, for the tile after the next, as soon as its product is formed.
//
// Work is cut by bytes, not by sequence: the tiles of all (sequence, head)
// items stand in one line, and each of the two workgroups a CU holds takes an
// equal piece of it, so that batches of mixed lengths end everywhere at once.
// A piece covers some items whole, which it writes, and parts of at most two,
// which a second launch joins.  Inside a workgroup the four waves take the
// item's row tiles and, if it has fewer than four, its tiles in turn; they
// join through LDS.
#pragma once

#include "attn_launch.h"

namespace tb {

constexpr int kAttnWaves = 4;  // waves of a workgroup, of both kernels

template <bool FP8>
struct RowOps;

template <>
struct RowOps<false> {
  typedef uint16_t Elem;
  static constexpr int kBlocks = 1;  // 32-position blocks per tile
  typedef bf16x8 V8;
};

template <>
struct RowOps<true> {
  typedef uint8_t Elem;
  static constexpr int kBlocks = 2;
  typedef f16x8 V8;
};

__device__ __forceinline__ f32x4 mfma16(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(const f16x8& a, const f16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

template <int D>
struct RowsShared {
  float max[kAttnWaves][16], sum[kAttnWaves][16];
  float o[kAttnWaves][16][D + 4];
};

// One (sequence, head) of the sequences with few rows, and its tiles in the
// line of all of them.  A sequence that sees nothing still has one (empty)
// tile, in which its rows are written.
struct RowsItem {
  int64_t start;  // of its first tile in the line
  int tiles;      // of the line: at least 1
  int b, head, rows;
  PagedSeq seq;
  PagedSpan span;
  int first_tile, count;  // the tiles that some row sees
};

struct RowsSeq {
  PagedSeq seq;
  PagedSpan span;
  TileSpan tiles;
  int rows;  // 0: not of this kind
};

__device__ __forceinline__ RowsSeq rows_seq(const tb_paged_attention_args& a, const AttnPlan& plan, int64_t b) {
  const tb_paged_cache& c = a.cache;
  RowsSeq r;
  r.seq = paged_seq(c.cu_q, c.kv_len, b, c.total_q, plan.capacity);
  const int n = r.seq.n < (int)c.max_q ? r.seq.n : (int)c.max_q;
  r.rows = plan.is_chunk((int64_t)n * plan.group) ? 0 : n * plan.group;
  r.span = paged_span(r.seq, 0, n - 1, a.window);
  r.tiles = tile_span(r.span, rows_positions(c.cache_dtype == TB_FP8));
  return r;
}

// tiles of the line for each head of the sequence
__device__ __forceinline__ int line_tiles(const RowsSeq& r) {
  return r.rows == 0 ? 0 : r.tiles.count > 1 ? r.tiles.count : 1;
}

// a value that is the same in every lane, in scalar registers
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ int64_t wave_sum64(int64_t v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return uniform64(v);
}

// Tiles in the line.  Whole waves call this and get the same answer.
__device__ __forceinline__ int64_t rows_total(const tb_paged_attention_args& a, const AttnPlan& plan) {
  int64_t n = 0;
  for (int64_t b = threadIdx.x & 63; b < a.cache.B; b += 64) n += line_tiles(rows_seq(a, plan, b));
  return wave_sum64(n) * a.cache.heads_kv;
}

// Tiles before sequence b in the line (b < B).
__device__ __forceinline__ int64_t rows_before(const tb_paged_attention_args& a, const AttnPlan& plan, int64_t b) {
  int64_t n = 0;
  for (int64_t x = threadIdx.x & 63; x < b; x += 64) n += line_tiles(rows_seq(a, plan, x));
  return wave_sum64(n) * a.cache.heads_kv;
}

// The item that holds tile `at` of the line (at < total).
__device__ __forceinline__ RowsItem rows_item_at(const tb_paged_attention_args& a, const AttnPlan& plan, int64_t at) {
  const int lane = threadIdx.x & 63, heads = a.cache.heads_kv;
  int64_t before = 0;
  RowsItem it;
  for (int64_t b0 = 0; b0 < a.cache.B; b0 += 64) {
    int64_t up = 0;  // inclusive prefix over the lanes
    if (b0 + lane < a.cache.B) up = (int64_t)line_tiles(rows_seq(a, plan, b0 + lane)) * heads;
    const int64_t own = up;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int64_t t = __shfl_up(up, m);
      if (lane >= m) up += t;
    }
    const uint64_t past = __ballot(before + up > at);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      it.start = uniform64(before + __shfl(up - own, l));
      it.b = __builtin_amdgcn_readfirstlane((int)b0 + l);
      break;
    }
    before = uniform64(before + __shfl(up, 63));
  }
  const RowsSeq r = rows_seq(a, plan, it.b);
  it.tiles = line_tiles(r);
  it.head = __builtin_amdgcn_readfirstlane((int)((at - it.start) / it.tiles));
  it.start += (int64_t)it.head * it.tiles;
  // the same in every lane: kept in scalar registers
  it.rows = __builtin_amdgcn_readfirstlane(r.rows);
  it.tiles = __builtin_amdgcn_readfirstlane(it.tiles);
  it.seq.row0 = uniform64(r.seq.row0);
  it.seq.n = __builtin_amdgcn_readfirstlane(r.seq.n);
  it.seq.keys = __builtin_amdgcn_readfirstlane(r.seq.keys);
  it.seq.first_pos = __builtin_amdgcn_readfirstlane(r.seq.first_pos);
  it.span.begin = __builtin_amdgcn_readfirstlane(r.span.begin);
  it.span.end = __builtin_amdgcn_readfirstlane(r.span.end);
  it.first_tile = __builtin_amdgcn_readfirstlane(r.tiles.first);
  it.count = __builtin_amdgcn_readfirstlane(r.tiles.count);
  return it;
}

// Tiles t0 .. t1 - 1 of an item: its output (slot < 0: they are all of it), or
// a part of it into the workspace's slot.
template <int D, bool FP8>
__device__ __forceinline__ void attn_rows_part(const tb_paged_attention_args& a, const AttnPlan& plan,
                                               const RowsItem& it, int t0, int t1, int64_t slot, RowsShared<D>& sm) {
  typedef RowOps<FP8> O;
  typedef typename O::Elem Elem;
  typedef typename O::V8 V8;
  constexpr int NB = O::kBlocks;          // 32-position blocks of a tile
  constexpr int T = rows_positions(FP8);  // positions of a tile
  constexpr int S = 2 * NB;               // 16-row score tiles of a tile
  constexpr int KL = D / 32 / NB;         // 16-byte loads of a key row per lane
  constexpr int DT = D / 16;              // 16-row tiles of O'

  const tb_paged_cache& c = a.cache;
  const int group = plan.group, head = it.head;
  const int64_t b = it.b;
  const PagedSeq& s = it.seq;
  const int nrows = it.rows, row_tiles = (nrows + 15) >> 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, q4 = lane >> 4;
  // the wave's row tile, and its place among the waves of that tile
  const int rt_bits = row_tiles == 1 ? 0 : row_tiles == 2 ? 1 : 2;
  const int rt = wave & ((1 << rt_bits) - 1), turn = wave >> rt_bits, step_t = kAttnWaves >> rt_bits;
  const int r0 = rt * kRowsTile;
  const bool wave_live = r0 < nrows;
  const int rl = r0 + kRowsTile - 1 < nrows ? r0 + kRowsTile - 1 : nrows - 1;  // last row
  const int j0 = (unsigned)(wave_live ? r0 : 0) / (unsigned)group, j1 = (unsigned)rl / (unsigned)group;
  const PagedSpan span = it.span;
  const int first_tile = it.first_tile;
  const int t_end = !wave_live ? 0 : t1 < it.count ? t1 : it.count;

  const int32_t* table = c.block_table + b * c.table_stride;
  const int shift = plan.shift, page = c.page;
  const int64_t page_step = (int64_t)c.heads_kv * page * D;
  const Elem* kc = static_cast<const Elem*>(c.k_cache) + (int64_t)head * page * D;
  const Elem* vc = static_cast<const Elem*>(c.v_cache) + (int64_t)head * page * D;

  // positions of the lane inside a tile: its key row (of score tile t, u):
  // krow + 8 t + 4 u, and its values: v0 .. v0 + 8 NB - 1
  const int krow = 8 * NB * (i16 >> 2) + (i16 & 3);
  const int v0 = 8 * NB * q4;

  // The page of position x, or -1 (none, or nobody sees it; its table entry is not read then).
  auto page_of = [&](int x) -> int {
    if ((x | (page - 1)) < span.begin || x >= span.end) return -1;
    return paged_page(table, c.table_width, c.n_pages, x >> shift);
  };
  struct Pages {
    int k, v;  // of the lane's keys and values
  };
  auto lookup = [&](int t) -> Pages {
    if (t >= t_end) return Pages{-1, -1};
    const int x0 = (first_tile + t) * T;
    return Pages{page_of(x0 + krow), page_of(x0 + v0)};
  };
  struct Tile {
    u32x4 k[S][KL], v[DT];
    int page;  // of the values
  };
  const int k_off = (krow & 15) * D + (16 / (int)sizeof(Elem)) * q4, v_off = i16 * page + (v0 & 15);
  auto load_keys = [&](Tile& x, int t, const Pages& pg) {
    if (t >= t_end) return;
    const int slot = ((first_tile + t) * T + (krow & ~15)) & (page - 1);
    const Elem* p = kc + (pg.k < 0 ? 0 : pg.k) * page_step + slot * D + k_off;
#pragma unroll
    for (int st = 0; st < S; ++st)
#pragma unroll
      for (int kk = 0; kk < KL; ++kk)
        x.k[st][kk] = *reinterpret_cast<const u32x4*>(p + (8 * (st >> 1) + 4 * (st & 1)) * D + 32 * NB * kk);
  };
  auto load_values = [&](Tile& x, int t, const Pages& pg) {
    x.page = pg.v;
    if (t >= t_end) return;
    const int slot = ((first_tile + t) * T + (v0 & ~15)) & (page - 1);
    const Elem* p = vc + (pg.v < 0 ? 0 : pg.v) * page_step + slot + v_off;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) x.v[dt] = *reinterpret_cast<const u32x4*>(p + 16 * dt * page);
  };

  int t = t0 + turn;
  Tile ta;
  const Pages pa = lookup(t);
  Pages ahead = lookup(t + step_t);

  // the lane's row
  const int r = r0 + i16;
  const bool row_live = r < nrows;
  const int tok = row_live ? (int)((unsigned)r / (unsigned)group) : 0;
  const int hq = head * group + (row_live ? r - tok * group : 0);
  const int pos = s.first_pos + tok;                                 // sees positions <= pos ..
  const int64_t low = a.window > 0 ? (int64_t)pos - a.window : -1;   // .. and > low
  bf16x8 q[D / 32];
  {
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (s.row0 + tok) * a.q_stride + (int64_t)hq * D;
#pragma unroll
    for (int kk = 0; kk < D / 32; ++kk) {
      // the d that lane group q4 of this step multiplies, as the key loads give them
      const int d = FP8 ? 64 * (kk / 2) + 16 * q4 + 8 * (kk % 2) : 32 * kk + 8 * q4;
      u32x4 w = {0u, 0u, 0u, 0u};
      if (row_live) w = *reinterpret_cast<const u32x4*>(qp + d);
      q[kk] = __builtin_bit_cast(bf16x8, w);
    }
  }
  const float scale2 = a.scale * kLog2e * (FP8 && c.k_scale ? c.k_scale[head] : 1.f);

  load_keys(ta, t, pa);
  load_values(ta, t, pa);

  float m = -__builtin_inff(), l = 0.f;
  f32x4 o[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) o[dt] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Tile t, held in `x`, which is loaded again for the tile after the next.
  auto step = [&](Tile& x, int t) {
    const int x0 = (first_tile + t) * T, pv = x.page;
    // looked up before that tile's loads: loads return in order, and the next
    // step waits for this one's answer only
    const Pages now = ahead;
    ahead = lookup(t + 2 * step_t);
    f32x4 sc[S];
#pragma unroll
    for (int st = 0; st < S; ++st) {
      sc[st] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < KL; ++kk) {
        if constexpr (FP8) {
          const u32x4 w = x.k[st][kk];
          sc[st] = mfma16(fp8_to_bf16(u32x2{w[0], w[1]}), q[2 * kk], sc[st]);
          sc[st] = mfma16(fp8_to_bf16(u32x2{w[2], w[3]}), q[2 * kk + 1], sc[st]);
        } else {
          sc[st] = mfma16(__builtin_bit_cast(bf16x8, x.k[st][kk]), q[kk], sc[st]);
        }
      }
    }
    load_keys(x, t + step_t, now);

    // scores in log2 units; what the row does not see is -inf.  The lane's
    // scores and its values are of the same positions, so of one page.
#pragma unroll
    for (int st = 0; st < S; ++st)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[st][e] *= scale2;
    // every row of the tile sees every position of it
    const bool full = __ballot(pv < 0) == 0 && x0 + T - 1 <= s.first_pos + j0 &&
                      (a.window <= 0 || x0 > (int64_t)s.first_pos + j1 - a.window);
    uint32_t seen = 0xffffffffu;  // bit 4 st + e
    if (!full) {
      seen = 0;
      const int64_t rel = (int64_t)x0 + v0;
      const int hi = row_live && pv >= 0 ? (int)(pos - rel < -1 ? -1 : pos - rel > 31 ? 31 : pos - rel) : -1;
      const int lo = (int)(low - rel < -1 ? -1 : low - rel > 31 ? 31 : low - rel);
#pragma unroll
      for (int st = 0; st < S; ++st)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int y = 8 * (st >> 1) + 4 * (st & 1) + e;
          const bool see = y <= hi && y > lo;
          seen |= (see ? 1u : 0u) << (4 * st + e);
          sc[st][e] = see ? sc[st][e] : -__builtin_inff();
        }
    }

    float top = sc[0][0];
#pragma unroll
    for (int st = 0; st < S; ++st)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, sc[st][e]);
    const float m_new = fmaxf(m, max_over_rows(top));
    const float base = m_new == -__builtin_inff() ? 0.f : m_new;
    const float alpha = exp2_fast(m - base);
    m = m_new;
    float sum = 0.f;
#pragma unroll
    for (int st = 0; st < S; ++st)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[st][e] = exp2_fast(sc[st][e] - base);
        sum += sc[st][e];
      }
    l = fmaf(l, alpha, sum);
    if (__ballot(alpha != 1.f) != 0) {
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[dt] *= alpha;
    }

    if (!full) {
      bool bad = false;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) bad = bad || (FP8 ? any_nonfinite_fp8(x.v[dt]) : any_nonfinite_bf16(x.v[dt]));
      if (__ballot(bad) != 0) {
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          f32x4 up = {0.f, 0.f, 0.f, 0.f}, down = up;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            V8 v, see;
#pragma unroll
            for (int e = 0; e < 8; ++e) see[e] = (seen >> (8 * nb + e)) & 1u ? 1.f : 0.f;
            if constexpr (FP8) v = fp8_to_f16(u32x2{x.v[dt][2 * nb], x.v[dt][2 * nb + 1]});
            else v = __builtin_bit_cast(bf16x8, x.v[dt]);
            const Nonfinite<V8> nf = take_nonfinite(v);
            up = mfma16(nf.up, see, up);
            down = mfma16(nf.down, see, down);
            if constexpr (!FP8) x.v[dt] = __builtin_bit_cast(u32x4, v);
          }
          if constexpr (FP8) x.v[dt] = drop_nonfinite_fp8(x.v[dt]);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[dt][e] += nonfinite_sum(up[e], down[e]);
          __builtin_amdgcn_sched_barrier(0);  // one at a time: this path is rare, its registers are not to count
        }
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      // Weights are rounded to 11 bits (fp16: every e4m3 value is exact in
      // it) or, for bf16 values, given as the sum of two bf16 numbers (16
      // bits): the matrix unit has room, and one bf16 would add an error as
      // large as the output's own rounding.
      V8 w, low_w;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float p = sc[2 * nb + (e >> 2)][e & 3];
        if constexpr (FP8) {
          w[e] = (_Float16)p;
        } else {
          w[e] = (__bf16)p;
          low_w[e] = (__bf16)(p - (float)w[e]);
        }
      }
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        if constexpr (FP8) {
          o[dt] = mfma16(fp8_to_f16(u32x2{x.v[dt][2 * nb], x.v[dt][2 * nb + 1]}), w, o[dt]);
        } else {
          const bf16x8 v = __builtin_bit_cast(bf16x8, x.v[dt]);
          o[dt] = mfma16(v, w, o[dt]);
          o[dt] = mfma16(v, low_w, o[dt]);
        }
      }
    }
    load_values(x, t + step_t, now);
  };
  while (t < t_end) {
    step(ta, t);
    t += step_t;
  }

  // the waves' sums joined: each scales its values to its row tile's common maximum
  l = sum_over_rows(l);
  if (q4 == 0) {
    sm.max[wave][i16] = m;
    sm.sum[wave][i16] = l;
  }
  __syncthreads();
  {
    float top = -__builtin_inff();
    for (int w = rt; w < kAttnWaves; w += 1 << rt_bits) top = fmaxf(top, sm.max[w][i16]);
    const float f = exp2_fast(m - (top == -__builtin_inff() ? 0.f : top));
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) *reinterpret_cast<f32x4*>(&sm.o[wave][i16][16 * dt + 4 * q4]) = o[dt] * f;
  }
  __syncthreads();
  constexpr int DL = D / 16;  // channels of a thread: 16 threads a row
  const int d0 = (threadIdx.x & 15) * DL;
  for (int k = 0; k < row_tiles; ++k) {
    const int x = threadIdx.x >> 4, row = 16 * k + x;
    if (row >= nrows) break;
    float top = -__builtin_inff(), total = 0.f;
    for (int w = k; w < kAttnWaves; w += 1 << rt_bits) top = fmaxf(top, sm.max[w][x]);
    const float base = top == -__builtin_inff() ? 0.f : top;
    f32x4 v[DL / 4];
#pragma unroll
    for (int e = 0; e < DL / 4; ++e) v[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int w = k; w < kAttnWaves; w += 1 << rt_bits) {
      total = fmaf(sm.sum[w][x], exp2_fast(sm.max[w][x] - base), total);
#pragma unroll
      for (int e = 0; e < DL / 4; ++e) v[e] += *reinterpret_cast<const f32x4*>(&sm.o[w][x][d0 + 4 * e]);
    }
    if (slot >= 0) {
      const int64_t pr = slot * plan.slot_rows + row;
      if (d0 == 0) plan.rows_stats[pr] = float2{top, total};
#pragma unroll
      for (int e = 0; e < DL / 4; ++e) *reinterpret_cast<f32x4*>(plan.rows_values + pr * D + d0 + 4 * e) = v[e];
    } else {
      const int otok = (unsigned)row / (unsigned)group;
      const int64_t at = (s.row0 + otok) * a.heads_q + head * group + (row - otok * group);
      const RowScale rs = row_scale(a, head, at, d0 == 0, top, total);
#pragma unroll
      for (int e = 0; e < DL / 4; ++e) write4(a, at * D + d0 + 4 * e, v[e], rs);
    }
  }
}

// Piece `block` of the items with few rows.
template <int D, bool FP8>
__device__ __forceinline__ void attn_rows(const tb_paged_attention_args& a, const AttnPlan& plan, unsigned block,
                                          RowsShared<D>& sm) {
  const int64_t total = rows_total(a, plan), per = plan.piece(total);
  int64_t at = (int64_t)block * per;
  const int64_t end = at + per < total ? at + per : total;
  bool first = true;
  while (at < end) {
    const RowsItem it = rows_item_at(a, plan, at);
    const int t0 = (int)(at - it.start);
    const int64_t past = it.start + it.tiles;
    const int t1 = (int)((past < end ? past : end) - it.start);
    attn_rows_part<D, FP8>(a, plan, it, t0, t1, t0 == 0 && t1 == it.tiles ? -1 : 2 * (int64_t)block + (first ? 0 : 1), sm);
    at = it.start + t1;
    first = false;
    if (at < end) __syncthreads();  // the next part writes the LDS that this one reads
  }
}

// Item `block` of B * heads_kv, in one part.
template <int D, bool FP8>
__device__ __forceinline__ void attn_rows_whole(const tb_paged_attention_args& a, const AttnPlan& plan, unsigned block,
                                                RowsShared<D>& sm) {
  const unsigned heads = (unsigned)a.cache.heads_kv;
  const RowsSeq r = rows_seq(a, plan, block / heads);
  if (r.rows == 0) return;
  const RowsItem it{0, line_tiles(r), (int)(block / heads), (int)(block % heads), r.rows, r.seq, r.span, r.tiles.first,
                    r.tiles.count};
  attn_rows_part<D, FP8>(a, plan, it, 0, it.tiles, -1, sm);
}

}  // namespace tb
