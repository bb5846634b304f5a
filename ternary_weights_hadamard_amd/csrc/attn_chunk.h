// Attention over the paged cache for many rows: chunks of prompts, and drafted
// tokens of many heads (include/tb.h, tb_paged_attention).
//
// Mathematics.  A wave keeps 32 rows (token, head of one key/value head) as
// the columns of S' = K Q' (v_mfma 32x32x16): a lane holds half of a row's
// scores, so a row's maximum is one exchange between two lanes, and with the
// positions behind the matrix rows of K permuted, the eight weights a lane
// forms of each 16 positions are, as they are, its operand of O' = V' P'.
// Weights never leave their lane.
//
// What bounds it: the matrix unit, the vector unit (scores -> weights) and the
// LDS reads of the operands take about as long as one another (for 64
// positions and 32 rows of 128: 1024 cycles of each), so the kernel lives from
// overlapping them: two workgroups of four waves per CU, a tile of 64
// positions of K and V double buffered in LDS and loaded by the
// global-to-LDS path while the tile before it is worked on.
#pragma once

#include "attn_rows.h"

namespace tb {

constexpr int kTile = kChunkPositions;
static_assert(kChunkTile == 32 * kAttnWaves && kTile == 64, "the lane layouts below");

__device__ __forceinline__ f32x16 mfma32(const bf16x8& a, const bf16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(const f16x8& a, const f16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

template <bool FP8>
struct ChunkOps;
template <>
struct ChunkOps<false> {
  typedef uint16_t Elem;
  typedef bf16x8 V8;
  static __device__ __forceinline__ __bf16 narrow(float x) { return (__bf16)x; }
};
template <>
struct ChunkOps<true> {  // e4m3 values are widened to fp16 in LDS, and weights have its 11 bits
  typedef uint8_t Elem;
  typedef f16x8 V8;
  static __device__ __forceinline__ _Float16 narrow(float x) { return (_Float16)x; }
};

// 16-byte chunks of the two tiles in LDS.  Row r of K (a position) has D / 8 of
// them, row r of V (a channel) kTile / 8; chunk c of a row lies at c ^ f(r), so
// that the lanes of a read, which take the same chunk of different rows, fall
// on different banks.
template <int D>
__device__ __forceinline__ int k_chunk(int row, int c) {
  return row * (D / 8) + (c ^ (row & (D / 8 - 1)));
}
__device__ __forceinline__ int v_chunk(int row, int c) { return row * (kTile / 8) + (c ^ ((row >> 1) & 7)); }

// Values that are not finite, in a tile that not every row sees all of (the
// products multiply every value with every row's weight, 0 where it does not
// see the position).  They are set to 0 in LDS.  Where some row sees one, it is
// first noted in bits which rows see a +inf (or NaN), and which a -inf (or NaN),
// in each channel: marks[row][D / 32][2], zero at the start; `marked` says that
// there are any.  All waves of the workgroup come here together, with the tile
// in v_lds and a barrier behind them.
//   x0, there   the tile's first position, and which of its runs of 16 exist
//   begin, end  the positions that some row sees
template <int D, bool FP8, int ROWS>
__device__ __forceinline__ void take_nonfinite_tile(u32x4* v_lds, uint32_t* marks, bool& marked, int x0, uint32_t there,
                                                    int begin, int end, int first_pos, int group, int r0, int nrows,
                                                    int64_t window) {
  constexpr int kThreads = 64 * kAttnWaves, kChunks = kTile * D / 8;
  typedef typename ChunkOps<FP8>::V8 V8;
  const int tid = threadIdx.x;
  int bad = 0;  // 1: some value is not finite, 2: at a position that some row sees
#pragma unroll 1
  for (int i = tid; i < kChunks; i += kThreads) {
    const u32x4 w = v_lds[i];
    if (!(FP8 ? any_nonfinite_f16(w) : any_nonfinite_bf16(w))) continue;
    const int row = i / (kTile / 8), x = x0 + (((i % (kTile / 8)) ^ ((row >> 1) & 7)) * 8);  // of the chunk: v_chunk
    bad |= x + 8 > begin && x < end ? 3 : 1;
  }
  if (!__syncthreads_or(bad)) return;
  if (__syncthreads_or(bad & 2)) {
    marked = true;
    // a thread has one row, and a share of the channels
    const int row = tid % ROWS, share = tid / ROWS;
    constexpr int kMine = D / (kThreads / ROWS);
    const bool live = r0 + row < nrows;
    const int64_t pos = (int64_t)first_pos + (int)((unsigned)(live ? r0 + row : r0) / (unsigned)group) - x0;
    const int64_t low = window > 0 ? pos - window : -1;
#pragma unroll 1
    for (int d = share * kMine; d < share * kMine + kMine; ++d) {
      uint32_t up = 0, down = 0;
#pragma unroll 1
      for (int ch = 0; ch < kTile / 8; ++ch) {
        const V8 v = __builtin_bit_cast(V8, v_lds[v_chunk(d, ch)]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = (float)v[e];
          const int x = 8 * ch + e;
          if (fabsf(f) < __builtin_inff() || !live || x > pos || x <= low || !((there >> (x >> 4)) & 1u)) continue;
          if (!(f < 0.f)) up = 1;
          if (!(f > 0.f)) down = 1;
        }
      }
      if (up | down) {
        uint32_t* at = marks + (row * (D / 32) + (d >> 5)) * 2;
        if (up) atomicOr(at, 1u << (d & 31));
        if (down) atomicOr(at + 1, 1u << (d & 31));
      }
    }
    __syncthreads();
  }
#pragma unroll 1
  for (int i = tid; i < kChunks; i += kThreads) {
    V8 v = __builtin_bit_cast(V8, v_lds[i]);
    take_nonfinite(v);
    v_lds[i] = __builtin_bit_cast(u32x4, v);
  }
  __syncthreads();
}

// What a row's marks add to its channels 32 dt + c .. + 3.
template <int D>
__device__ __forceinline__ f32x4 marked_sum(const uint32_t* marks, int row, int dt, int c) {
  const uint32_t up = marks[(row * (D / 32) + dt) * 2] >> c, down = marks[(row * (D / 32) + dt) * 2 + 1] >> c;
  f32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = nonfinite_sum((up >> e) & 1u ? 1.f : 0.f, (down >> e) & 1u ? 1.f : 0.f);
  return r;
}

// Tiles t_begin .. t_stop - 1 of an item: its output (slot < 0: they are all of
// it), or a part of it into the workspace's slot.
template <int D, bool FP8>
__device__ __forceinline__ void attn_chunk_part(const tb_paged_attention_args& a, const AttnPlan& plan,
                                                const LineItem& it, int t_begin, int t_stop, int64_t slot,
                                                const AttnShared& sm) {
  typedef typename ChunkOps<FP8>::Elem Elem;
  typedef typename ChunkOps<FP8>::V8 V8;
  constexpr int KK = D / 16;   // steps of a score tile
  constexpr int DT = D / 32;   // 32-channel tiles of O'
  constexpr int kWaves = kAttnWaves, kRows = kChunkTile;

  const tb_paged_cache& c = a.cache;
  const int group = plan.group, head = it.head, nrows = it.seq.rows;
  const PagedSeq& s = it.seq.seq;
  const PagedSpan& span = it.span;
  const int r0 = it.rt * kRows;
  const int r_last = r0 + kRows - 1 < nrows ? r0 + kRows - 1 : nrows - 1;
  const int j_first = uniform((unsigned)r0 / (unsigned)group), j_last = uniform((unsigned)r_last / (unsigned)group);
  const int first_tile = it.held.first, t_end = t_stop < it.held.count ? t_stop : it.held.count;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int i32 = lane & 31, half = lane >> 5;

  // the lane's row, and its wave's first and last
  const int r = r0 + wave * 32 + i32;
  const bool row_live = r < nrows;
  const int tok = row_live ? (int)((unsigned)r / (unsigned)group) : 0;
  const int hq = head * group + (row_live ? r - tok * group : 0);
  const int pos = s.first_pos + tok;
  const int64_t low = a.window > 0 ? (int64_t)pos - a.window : -1;
  const int w_first = r0 + wave * 32 < nrows ? r0 + wave * 32 : nrows - 1;
  const int w_last = w_first + 31 < nrows ? w_first + 31 : nrows - 1;
  const int pos_first = uniform(s.first_pos + (int)((unsigned)w_first / (unsigned)group));
  const int pos_last = uniform(s.first_pos + (int)((unsigned)w_last / (unsigned)group));
  // and of the workgroup
  const int all_first = s.first_pos + j_first, all_last = s.first_pos + j_last;

  // scores are scaled by |scale|; its sign goes into the queries.  A scale of
  // 0 is taken as the smallest number, so that an unseen -inf stays one.
  float scale2 = a.scale * kLog2e * (FP8 && c.k_scale ? c.k_scale[head] : 1.f);
  const uint32_t flip = scale2 < 0.f ? 0x80008000u : 0u;
  scale2 = fmaxf(fabsf(scale2), 1.17549435e-38f);
  bf16x8 q[KK];
  {
    const uint16_t* qp =
        static_cast<const uint16_t*>(a.q) + (s.row0 + tok) * a.q_stride + (int64_t)hq * D + 8 * half;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      u32x4 w = {0u, 0u, 0u, 0u};
      if (row_live) w = *reinterpret_cast<const u32x4*>(qp + 16 * kk);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] ^= flip;
      q[kk] = __builtin_bit_cast(bf16x8, w);
    }
  }

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
  auto stage = [&](int t, int pages, u32x4* k_to, u32x4* v_to) {
    const int x0 = (first_tile + t) * kTile;
    const Elem* vp = vc + (pages < 0 ? 0 : pages) * page_step + ((x0 + 16 * v_run) & (c.page - 1)) + v_off;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int run = (i * kStep + __builtin_amdgcn_readfirstlane(k_row)) >> 4;
      const int page = run_page(pages, run);
      const Elem* kp = kc + (page < 0 ? 0 : page) * page_step + (int64_t)((x0 + 16 * run) & (c.page - 1)) * D;
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

  // matrix row m of a score tile stands for position key(m) of its 32: a
  // lane's score registers 0..7 are then positions 8 half + 0..7, 8..15 are 16 more
  const int key = 16 * (i32 >> 4) + 8 * ((i32 >> 2) & 1) + 4 * ((i32 >> 3) & 1) + (i32 & 3);

  float m = -__builtin_inff(), l = 0.f;  // maximum (log2 units) that the weights are relative to, and the lane's sum
  f32x16 o[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[dt][e] = 0.f;

  bool marked = false;
#pragma unroll
  for (int i = 0; i < kRows * D / 16 / (64 * kWaves); ++i) sm.marks[i * 64 * kWaves + tid] = 0u;  // a barrier follows
  int pages = lookup(t_begin), pages_next = lookup(t_begin + 1);
  if (t_begin < t_end) {
    stage(t_begin, pages, sm.buffer[0], sm.buffer[1]);
    widen(sm.buffer[0], sm.buffer[1]);
  }
  // Tile t, in k_lds and v_lds, while tile t + 1 is loaded into k_to and v_to.
  // The four are arrays of their own, and which is which is known when this is
  // compiled: the compiler then knows that reading the one does not wait for
  // the loads into the other.
  auto step = [&](int t, u32x4* k_lds, u32x4* v_lds, u32x4* k_to, u32x4* v_to) {
    __builtin_amdgcn_s_waitcnt(0);  // this wave's share of the tile is in LDS
    __syncthreads();
    if (t + 1 < t_end) stage(t + 1, pages_next, k_to, v_to);
    const int pages_after = lookup(t + 2);
    const int x0 = (first_tile + t) * kTile;
    uint32_t there = 0xfu;  // which of the tile's runs exist
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (run_page(pages, g) < 0) there &= ~(1u << g);
    // does any row of the wave see any of it; do all of the workgroup's see all of it
    const bool any = x0 <= pos_last && (a.window <= 0 || x0 + kTile - 1 > pos_first - a.window);
    const bool all_full = there == 0xfu && x0 + kTile - 1 <= all_first && (a.window <= 0 || x0 > all_last - a.window);
    f32x16 sc[2];
    if (any) {
#pragma unroll
      for (int e = 0; e < 16; ++e) sc[0][e] = sc[1][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          sc[u] = mfma32(__builtin_bit_cast(bf16x8, k_lds[k_chunk<D>(32 * u + key, 2 * kk + half)]), q[kk], sc[u]);

      // The lane's scores: register 8 k + e of tile u is position 32 u + 16 k + 8 half + e.
      const bool full = there == 0xfu && x0 + kTile - 1 <= pos_first && (a.window <= 0 || x0 > pos_last - a.window);
      if (!full) {
        const int64_t rel = (int64_t)x0 + 8 * half;
        const int hi = row_live ? (int)(pos - rel < -1 ? -1 : pos - rel > 63 ? 63 : pos - rel) : -1;
        const int lo = (int)(low - rel < -1 ? -1 : low - rel > 63 ? 63 : low - rel);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int x = 32 * u + 16 * (e >> 3) + (e & 7);
            const bool see = x <= hi && x > lo && ((there >> (2 * u + (e >> 3))) & 1u);
            sc[u][e] = see ? sc[u][e] : -__builtin_inff();
          }
      }

      float top = sc[0][0];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, sc[u][e]);
      float t0, t1;
      swap_halves(top, t0, t1);
      top = fmaxf(t0, t1) * scale2;
      // The weights stay relative to an older maximum while the new one is
      // less than 2^8 above it: nothing is rounded more (they are at most 2^8),
      // and the values' sums are rarely rescaled.
      if (__ballot(top > m + 8.f) != 0) {
        const float m_new = fmaxf(m, top);
        const float alpha = m == -__builtin_inff() ? 1.f : exp2_fast(m - m_new);
        m = m_new;
        l *= alpha;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[dt][e] *= alpha;
      }
      const float base = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          sc[u][e] = exp2_fast(fmaf(sc[u][e], scale2, -base));
          l += sc[u][e];
        }
    }

    if (!all_full)
      take_nonfinite_tile<D, FP8, kRows>(v_lds, sm.marks, marked, x0, there, span.begin, span.end, s.first_pos, group, r0,
                                         nrows, a.window);

    if (any) {
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        V8 w;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = ChunkOps<FP8>::narrow(sc[kb >> 1][8 * (kb & 1) + e]);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
          o[dt] = mfma32(__builtin_bit_cast(V8, v_lds[v_chunk(32 * dt + i32, 2 * kb + half)]), w, o[dt]);
      }
    }
    pages = pages_next;
    pages_next = pages_after;
    widen(k_to, v_to);
  };
  for (int t = t_begin; t < t_end; t += 2) {
    step(t, sm.buffer[0], sm.buffer[1], sm.buffer[2], sm.buffer[3]);
    if (t + 1 < t_end) step(t + 1, sm.buffer[2], sm.buffer[3], sm.buffer[0], sm.buffer[1]);
  }

  // the row's sum, and its output: register 4 j + e of tile dt is channel 32 dt + 8 j + 4 half + e
  {
    float a0, a1;
    swap_halves(l, a0, a1);
    l = a0 + a1;
  }
  if (!row_live) return;
  if (marked) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4 x = marked_sum<D>(sm.marks, r - r0, dt, 8 * j + 4 * half);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[dt][4 * j + e] += x[e];
      }
  }
  const int64_t at = (s.row0 + tok) * a.heads_q + hq;
  if (slot >= 0) {
    const int64_t pr = slot * kRows + (r - r0);
    if (half == 0) plan.chunk_line.stats[pr] = float2{m, l};
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<f32x4*>(plan.chunk_line.values + pr * D + 32 * dt + 8 * j + 4 * half) =
            f32x4{o[dt][4 * j], o[dt][4 * j + 1], o[dt][4 * j + 2], o[dt][4 * j + 3]};
    return;
  }
  const RowScale rs = row_scale(a, head, at, half == 0, m, l);
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      write4(a, at * D + 32 * dt + 8 * j + 4 * half,
             f32x4{o[dt][4 * j], o[dt][4 * j + 1], o[dt][4 * j + 2], o[dt][4 * j + 3]}, rs);
}

}  // namespace tb
