// Attention over the paged cache for chunks whose row tiles fill the GPU
// (include/tb.h, tb_paged_attention): the chunk kernel's mathematics
// (attn_chunk.h) with 64 rows a wave.
//
// What bounds it: the matrix unit, if the vector work of turning scores into
// weights runs beside it.  Two waves of 32 rows on a SIMD do not manage that
// (matrix unit busy 35 % of the time, vector unit 41 %, one after the other: a
// wave waits for its operands from LDS, for its products, or for the other
// wave).  So one wave has two halves of 32 rows, A and B, and all of a SIMD's
// registers, and the instruction stream itself interleaves: while A's scores of
// 32 positions become weights, B's products are formed (its scores of these
// positions, then its values' sums of those before), then the other way round.
// The maximum of a half's new scores is taken beside its values' products too;
// what is left outside is the decision to rescale.  K and V are three tiles
// deep in LDS, and a workgroup has 256 rows.
#pragma once

#include "attn_chunk.h"

namespace tb {

// 32 rows of a wave.
template <int D, bool FP8>
struct WideHalf {
  bf16x8 q[D / 16];
  f32x16 sc, o[D / 32];
  typename ChunkOps<FP8>::V8 w[2];
  float m, base, l;  // maximum (log2 units), the same or 0, the lane's sum
  float top;         // of the lane's new scores, if all are seen
  int pos, hq, tok;
  int64_t low;
  bool live;
  int pos_first, pos_last;
};

template <int D, bool FP8>
__device__ __forceinline__ void attn_wide_part(const tb_paged_attention_args& a, const AttnPlan& plan,
                                               const LineItem& it, const WideShared& sm) {
  typedef typename ChunkOps<FP8>::Elem Elem;
  typedef typename ChunkOps<FP8>::V8 V8;
  typedef WideHalf<D, FP8> Half;
  constexpr int KK = D / 16;   // steps of a score tile
  constexpr int DT = D / 32;   // 32-channel tiles of O'
  constexpr int kChunks = kTile * D / 8;  // 16-byte chunks of a tile of K, and of V
  constexpr int kWaves = kAttnWaves, kRows = kWideTile;

  const tb_paged_cache& c = a.cache;
  const int group = plan.group, head = it.head, nrows = it.seq.rows;
  const PagedSeq& s = it.seq.seq;
  const PagedSpan& span = it.span;
  const int r0 = it.rt * kRows;
  const int r_last = r0 + kRows - 1 < nrows ? r0 + kRows - 1 : nrows - 1;
  const int all_first = s.first_pos + uniform((unsigned)r0 / (unsigned)group);
  const int all_last = s.first_pos + uniform((unsigned)r_last / (unsigned)group);
  const int first_tile = it.held.first, t_end = it.held.count;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int i32 = lane & 31, half = lane >> 5;

  float scale2 = a.scale * kLog2e * (FP8 && c.k_scale ? c.k_scale[head] : 1.f);
  const uint32_t flip = scale2 < 0.f ? 0x80008000u : 0u;  // as in attn_chunk.h
  scale2 = fmaxf(fabsf(scale2), 1.17549435e-38f);

  Half ha, hb;
  auto start = [&](Half& h, int first_row) {
    const int r = r0 + first_row + i32;
    h.live = r < nrows;
    h.tok = h.live ? (int)((unsigned)r / (unsigned)group) : 0;
    h.hq = head * group + (h.live ? r - h.tok * group : 0);
    h.pos = s.first_pos + h.tok;
    h.low = a.window > 0 ? (int64_t)h.pos - a.window : -1;
    const int w_first = r0 + first_row < nrows ? r0 + first_row : nrows - 1;
    const int w_last = w_first + 31 < nrows ? w_first + 31 : nrows - 1;
    h.pos_first = uniform(s.first_pos + (int)((unsigned)w_first / (unsigned)group));
    h.pos_last = uniform(s.first_pos + (int)((unsigned)w_last / (unsigned)group));
    const uint16_t* qp =
        static_cast<const uint16_t*>(a.q) + (s.row0 + h.tok) * a.q_stride + (int64_t)h.hq * D + 8 * half;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      u32x4 w = {0u, 0u, 0u, 0u};
      if (h.live) w = *reinterpret_cast<const u32x4*>(qp + 16 * kk);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] ^= flip;
      h.q[kk] = __builtin_bit_cast(bf16x8, w);
    }
    h.m = -__builtin_inff();
    h.base = h.l = h.top = 0.f;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int e = 0; e < 16; ++e) h.o[dt][e] = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) h.w[k][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) h.sc[e] = 0.f;
  };

  const int32_t* table = c.block_table + it.b * c.table_stride;
  const int shift = plan.shift;
  const int64_t page_elems = (int64_t)c.page * D, page_step = (int64_t)c.heads_kv * page_elems;
  const Elem* kc = static_cast<const Elem*>(c.k_cache) + head * page_elems;
  const Elem* vc = static_cast<const Elem*>(c.v_cache) + head * page_elems;

  // Staging.  bf16: a wave moves whole kilobytes from global memory to LDS,
  // lane i to the i-th 16 bytes, so the lanes read permuted chunks of their
  // rows.  8-bit: 16 values a lane through registers, widened on the way.
  //
  // A tile is four runs of 16 positions, each in one page.  What a lane loads
  // of V lies in run v_run, the same for all its loads, so it looks up that
  // run's page (-1: none, or nobody sees it; its entry is not read then), and
  // holder(g) is a lane that thereby holds run g's.  What a wave loads of K with one
  // instruction lies in one run.
  constexpr int kPer = FP8 ? 16 : 8;                               // positions (or channels) of a 16-byte load
  constexpr int kLoads = kTile * D / kPer / (64 * kWaves);         // loads of a lane, for K and for V
  constexpr int kStep = FP8 ? 64 * kWaves / (D / 16) : 64 * kWaves / (D / 8);        // rows of K between them
  constexpr int vStep = 64 * kWaves / (kTile / kPer);              // rows of V between them
  const int tid = wave * 64 + lane;
  const int k_row = tid / (D / kPer), v_row = tid / (kTile / kPer);  // of the first load
  const int k_ch = FP8 ? tid % (D / 16) : (tid % (D / 8)) ^ (k_row & (D / 8 - 1));
  const int v_ch = FP8 ? tid % 4 : (tid % 8) ^ ((v_row >> 1) & 7);
  const int v_run = FP8 ? v_ch : v_ch >> 1;
  const int k_off = (k_row & 15) * D + k_ch * kPer;                 // inside a run
  const int v_off = v_row * c.page + (v_ch * kPer & 15);
  auto lookup = [&](int t) -> int {
    const int x = (first_tile + t) * kTile + 16 * v_run;
    if (t >= t_end || (x | (c.page - 1)) < span.begin || x >= span.end) return -1;
    return paged_page(table, c.table_width, c.n_pages, x >> shift);
  };
  auto holder = [&](int g) { return FP8 ? g : 2 * g ^ 4 * (wave & 1); };  // bf16: row v_row of lanes 0..7 is 8 wave
  auto run_page = [&](int pages, int g) { return __builtin_amdgcn_readlane(pages, holder(g)); };
  u32x4 kr[FP8 ? kLoads : 1], vr[FP8 ? kLoads : 1];
  // K of one tile and V of another
  auto stage = [&](int tk, int pages_k, u32x4* k_to, int tv, int pages_v, u32x4* v_to) {
    const int xk = (first_tile + tk) * kTile, xv = (first_tile + tv) * kTile;
    const Elem* vp = vc + (pages_v < 0 ? 0 : pages_v) * page_step + ((xv + 16 * v_run) & (c.page - 1)) + v_off;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int run = (i * kStep + __builtin_amdgcn_readfirstlane(k_row)) >> 4;
      const int page = run_page(pages_k, run);
      const Elem* kp = kc + (page < 0 ? 0 : page) * page_step + (int64_t)((xk + 16 * run) & (c.page - 1)) * D;
      if constexpr (FP8) {
        kr[i] = *reinterpret_cast<const u32x4*>(kp + k_off);
        vr[i] = *reinterpret_cast<const u32x4*>(vp + i * vStep * c.page);
      } else {
        const int at = i * 64 * kWaves + wave * 64;  // the wave's first chunk
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t*)(kp + k_off),
                                         (__attribute__((address_space(3))) uint32_t*)&k_to[at], 16, 0, 0);
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) uint32_t*)(vp + i * vStep * c.page),
            (__attribute__((address_space(3))) uint32_t*)&v_to[at], 16, 0, 0);
      }
    }
  };
  auto widen = [&](u32x4* k_to, u32x4* v_to) {  // 8-bit: the staged registers into LDS
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int kw = i * kStep + k_row, vw = i * vStep + v_row;
        k_to[k_chunk<D>(kw, 2 * k_ch)] = __builtin_bit_cast(u32x4, fp8_to_bf16(u32x2{kr[i][0], kr[i][1]}));
        k_to[k_chunk<D>(kw, 2 * k_ch + 1)] = __builtin_bit_cast(u32x4, fp8_to_bf16(u32x2{kr[i][2], kr[i][3]}));
        v_to[v_chunk(vw, 2 * v_ch)] = __builtin_bit_cast(u32x4, fp8_to_f16(u32x2{vr[i][0], vr[i][1]}));
        v_to[v_chunk(vw, 2 * v_ch + 1)] = __builtin_bit_cast(u32x4, fp8_to_f16(u32x2{vr[i][2], vr[i][3]}));
      }
    }
  };

  const int key = 16 * (i32 >> 4) + 8 * ((i32 >> 2) & 1) + 4 * ((i32 >> 3) & 1) + (i32 & 3);  // as in attn_chunk.h

  // Whether all rows of a half see all of a tile; and if not, what the lane's
  // row sees: bit 16 u + 8 k + e is position 32 u + 16 k + 8 half + e.
  auto sees_all = [&](const Half& h, int x0, uint32_t there) {
    return there == 0xfu && x0 + kTile - 1 <= h.pos_first && (a.window <= 0 || x0 > (int64_t)h.pos_last - a.window);
  };
  auto seen_of = [&](const Half& h, int x0, uint32_t there) -> uint32_t {
    const int64_t rel = (int64_t)x0 + 8 * half;
    const int hi = h.live ? (int)(h.pos - rel < -1 ? -1 : h.pos - rel > 63 ? 63 : h.pos - rel) : -1;
    const int lo = (int)(h.low - rel < -1 ? -1 : h.low - rel > 63 ? 63 : h.low - rel);
    uint32_t seen = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // eight positions 16 k .. 16 k + 7 of the lane: those above lo and up to hi
      const int n = hi - 16 * k < -1 ? 0 : hi - 16 * k > 7 ? 8 : hi - 16 * k + 1;
      const int f = lo - 16 * k < -1 ? 0 : lo - 16 * k > 7 ? 8 : lo - 16 * k + 1;
      const uint32_t bits = ((1u << n) - 1u) & ~((1u << f) - 1u) & 0xffu;
      seen |= ((there >> k) & 1u ? bits : 0u) << (8 * k);
    }
    return seen;
  };

  // New scores of a half (32 positions: part u of the tile at x0): what its rows
  // do not see out, the maximum, and the values' sums rescaled if it has grown
  // by more than 2^8.
  auto settle = [&](Half& h, int u, int x0, uint32_t there) {
    float top = h.top;
    if (!sees_all(h, x0, there)) {
      const uint32_t seen = seen_of(h, x0, there) >> (16 * u);
      top = -__builtin_inff();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        h.sc[e] = (seen >> e) & 1u ? h.sc[e] : -__builtin_inff();
        top = fmaxf(top, h.sc[e]);
      }
    }
    float t0, t1;
    swap_halves(top, t0, t1);
    top = fmaxf(t0, t1) * scale2;
    if (__ballot(top > h.m + 8.f) != 0) {
      const float m_new = fmaxf(h.m, top);
      const float alpha = h.m == -__builtin_inff() ? 1.f : exp2_fast(h.m - m_new);
      h.m = m_new;
      h.base = m_new == -__builtin_inff() ? 0.f : m_new;
      h.l *= alpha;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int e = 0; e < 16; ++e) h.o[dt][e] *= alpha;
    }
  };

  // One half's scores become its weights beside the other half's products: its
  // scores of the keys of part uk in k_lds, and the sums of the values of part
  // uv in v_lds with its weights.  Straight-line code, a few vector
  // instructions for each product.
  auto beside = [&](Half& e, Half& g, const u32x4* k_lds, int uk, const u32x4* v_lds, int uv) {
    static_assert(2 * DT == KK, "as many products of values as of keys");
#pragma unroll
    for (int x = 0; x < 16; ++x) g.sc[x] = 0.f;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
      g.sc = mfma32(__builtin_bit_cast(bf16x8, k_lds[k_chunk<D>(32 * uk + key, 2 * kk + half)]), g.q[kk], g.sc);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
        g.o[dt] = mfma32(__builtin_bit_cast(V8, v_lds[v_chunk(32 * dt + i32, 2 * (2 * uv + kb) + half)]), g.w[kb], g.o[dt]);
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const float p = exp2_fast(fmaf(e.sc[x], scale2, -e.base));
      sum[x & 1] += p;
      e.w[x >> 3][x & 7] = ChunkOps<FP8>::narrow(p);
    }
    e.l += sum[0] + sum[1];
    float top = g.sc[0];
#pragma unroll
    for (int x = 1; x < 16; ++x) top = fmaxf(top, g.sc[x]);
    g.top = top;
    // the order: operands from LDS a few products ahead, and vector work beside each product
    constexpr int kAhead = 6, kBeside = 80 / (2 * KK) + 1;
    __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
    for (int i = 0; i < 2 * KK; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < 2 * KK - kAhead) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, kBeside, 0);
    }
  };

  bool marked = false;
#pragma unroll
  for (int i = 0; i < kRows * D / 16 / (64 * kWaves); ++i) sm.marks[i * 64 * kWaves + tid] = 0u;  // a barrier follows
  int p0 = lookup(0), p1 = lookup(1);
  start(ha, wave * 64);
  start(hb, wave * 64 + 32);
  if (t_end > 0) {
#pragma unroll
    for (int i = 0; i < kChunks / (64 * kWaves); ++i)  // B's first sums are of no tile: weights and values 0
      sm.v[2][i * 64 * kWaves + tid] = u32x4{0u, 0u, 0u, 0u};
    stage(0, p0, sm.k[0], 0, p0, sm.v[0]);
    widen(sm.k[0], sm.v[0]);
    if (t_end > 1) {
      stage(1, p1, sm.k[1], 0, p0, sm.v[0]);  // V again: the same bytes
      widen(sm.k[1], sm.v[0]);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
      ha.sc = mfma32(__builtin_bit_cast(bf16x8, sm.k[0][k_chunk<D>(key, 2 * kk + half)]), ha.q[kk], ha.sc);
    ha.top = ha.sc[0];
#pragma unroll
    for (int x = 1; x < 16; ++x) ha.top = fmaxf(ha.top, ha.sc[x]);
  }
  int p2 = lookup(2);
  // Tile t: K of t in k0, of t + 1 in k1, and t + 2 goes to k2; V of t - 1 in
  // v2, of t in v0, and t + 1 goes to v1.  A is half a tile ahead of B.
  auto step = [&](int t, u32x4* k0, u32x4* k1, u32x4* k2, u32x4* v0, u32x4* v1, u32x4* v2) {
    __builtin_amdgcn_s_waitcnt(0);  // this wave's share of what was staged a tile ago is in LDS
    __syncthreads();
    if (t + 1 < t_end) stage(t + 2 < t_end ? t + 2 : t + 1, t + 2 < t_end ? p2 : p1, k2, t + 1, p1, v1);
    const int p3 = lookup(t + 3);
    const int x0 = (first_tile + t) * kTile;
    uint32_t there = 0xfu;
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (run_page(p0, g) < 0) there &= ~(1u << g);
    if (!(there == 0xfu && x0 + kTile - 1 <= all_first && (a.window <= 0 || x0 > (int64_t)all_last - a.window)))
      take_nonfinite_tile<D, FP8, kRows>(v0, sm.marks, marked, x0, there, span.begin, span.end, s.first_pos, group, r0,
                                         nrows, a.window);
    settle(ha, 0, x0, there);
    beside(ha, hb, k0, 0, v2, 1);
    settle(hb, 0, x0, there);
    beside(hb, ha, k0, 1, v0, 0);
    settle(ha, 1, x0, there);
    beside(ha, hb, k0, 1, v0, 0);
    settle(hb, 1, x0, there);
    beside(hb, ha, k1, 0, v0, 1);  // past the last tile: scores of what lies in k1, not used
    if (t + 1 < t_end) widen(k2, v1);
    p0 = p1;
    p1 = p2;
    p2 = p3;
  };
  for (int t = 0; t < t_end; t += 3) {
    step(t, sm.k[0], sm.k[1], sm.k[2], sm.v[0], sm.v[1], sm.v[2]);
    if (t + 1 < t_end) step(t + 1, sm.k[1], sm.k[2], sm.k[0], sm.v[1], sm.v[2], sm.v[0]);
    if (t + 2 < t_end) step(t + 2, sm.k[2], sm.k[0], sm.k[1], sm.v[2], sm.v[0], sm.v[1]);
  }
  // B's sums of the last 32 positions
  auto finish = [&](const u32x4* v_lds) {
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
        hb.o[dt] = mfma32(__builtin_bit_cast(V8, v_lds[v_chunk(32 * dt + i32, 2 * (2 + kb) + half)]), hb.w[kb], hb.o[dt]);
  };
  if (t_end > 0) {
    if (t_end % 3 == 1) finish(sm.v[0]);
    else if (t_end % 3 == 2) finish(sm.v[1]);
    else finish(sm.v[2]);
  }

  auto write = [&](Half& h, int row) {
    float a0, a1;
    swap_halves(h.l, a0, a1);
    const float l = a0 + a1;
    if (!h.live) return;
    if (marked) {
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 x = marked_sum<D>(sm.marks, row, dt, 8 * j + 4 * half);
#pragma unroll
          for (int e = 0; e < 4; ++e) h.o[dt][4 * j + e] += x[e];
        }
    }
    const int64_t at = (s.row0 + h.tok) * a.heads_q + h.hq;
    const RowScale rs = row_scale(a, head, at, half == 0, h.m, l);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        write4(a, at * D + 32 * dt + 8 * j + 4 * half,
               f32x4{h.o[dt][4 * j], h.o[dt][4 * j + 1], h.o[dt][4 * j + 2], h.o[dt][4 * j + 3]}, rs);
  };
  write(ha, wave * 64 + i32);
  write(hb, wave * 64 + 32 + i32);
}

}  // namespace tb
