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
// What bounds it: a wave's own stream.  For 32 positions and 32 rows of 128
// channels the products take 512 cycles of the matrix unit and the weights
// about 450 of the vector unit, and two waves on a SIMD do not overlap the two
// by themselves (as two phases a tile, the matrix unit was busy 35 % of the time
// and the vector unit 41 %, one after the other).  So the instruction stream
// interleaves them: beside each product of the next 32 positions' scores two of
// these scores become weights, and beside the products of these positions'
// values the maximum of the next scores is taken; the loads of later tiles go
// out between them.  Of a tile's 4600 cycles a wave spends 2000 there, 700 in
// deciding to rescale, and the rest waiting for the other waves and looking
// pages up.  Tiles of 64 positions of K and V are double buffered in LDS by the
// memory-to-LDS path, each loaded one tile ahead; two workgroups of four waves
// share a CU.  4 x up to 2048 tokens over 2048..8192, 40 heads, 8
// key/value heads: 479 GFLOP in 500 us, 958 TFLOP/s (a large library product:
// 1255), 525 us in the first twenty calls, before the clock has risen; in e4m3
// 540 us, in pages of 16 602 us.  2 x 777 tokens over 6000 in a window of 1000,
// 16 heads of 64 in e4m3: 35.3 us.
#pragma once

#include <type_traits>

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

// 16 bytes of each active lane, from page + step + lane_at, to its place in the
// 1024 bytes at `to` in LDS; `page` and `step` are the same in every lane.  As
// a buffer load: behind global_load_lds the compiler cannot tell what a wait
// for LDS has to wait for, and waits for all of it every time (four times in
// 16 products, each time until the newest operand has come).
__device__ __forceinline__ void load_lds16(const void* page, int bytes, int lane_at, int step, u32x4* to) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kWord3 = 0x00020000;  // the 32-bit data format that raw loads need
  const __amdgpu_buffer_rsrc_t from = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(page), (short)0, bytes, kWord3);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, lane_at, step, 0, 0);
#endif
}

// Until at most N of the wave's loads are still on their way.
template <int N>
__device__ __forceinline__ void wait_loads() {
  // vmcnt: bits 3..0 and 15..14; the other counters are not waited for
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
}

// Weights are relative to weight_reference<kRoom> of a maximum that may lag
// behind the row's by 2^kSlack, so they are at most 2^(kRoom + kSlack).  For
// fp16 the two share its range: more slack is less room for small weights, less
// is more rescaling (the windowed chunk above, measured together: 37.9 us with a
// slack of 8, 38.5 with 4, 39.5 with 2).
template <bool FP8>
struct ChunkOps;
template <>
struct ChunkOps<false> {  // weights have bf16's 8 bits: as two bf16 (few rows) there would be half as many products again
  typedef uint16_t Elem;
  typedef bf16x8 V8;
  static constexpr int kRoom = 0, kSlack = 8;
  static __device__ __forceinline__ __bf16 narrow(float x) { return (__bf16)x; }
};
template <>
struct ChunkOps<true> {  // e4m3 values are widened to fp16 in LDS, and weights have its 11 bits
  typedef uint8_t Elem;
  typedef f16x8 V8;
  static constexpr int kRoom = 11, kSlack = 4;  // full precision down to 2^-25 of the largest weight
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

// Its argument is in vector registers at this point of the program, and may
// have changed: what makes it cannot be moved behind, what uses it not before.
template <typename T>
__device__ __forceinline__ void hold(T& x) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(x));
#else
  (void)x;
#endif
}

// The two low bits of x that are set in some lane of the workgroup, in every
// lane; a barrier.  Between two calls there has to be another.
// (__syncthreads_or counts lanes in three dimensions, in registers that the
// compiler keeps through the loop over the tiles: with it values are spilled.)
__device__ __forceinline__ int workgroup_bits(int x, int* of_wave) {
  of_wave[threadIdx.x >> 6] = (__ballot(x & 1) != 0 ? 1 : 0) | (__ballot(x & 2) != 0 ? 2 : 0);
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kAttnWaves; ++w) all |= of_wave[w];
  return uniform(all);
}

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
__device__ __forceinline__ void take_nonfinite_tile(u32x4* v_lds, const AttnShared& sm, bool& marked, int x0,
                                                    uint32_t there, int begin, int end, int first_pos, int group, int r0,
                                                    int nrows, int64_t window) {
  constexpr int kThreads = 64 * kAttnWaves, kChunks = kTile * D / 8;
  typedef typename ChunkOps<FP8>::V8 V8;
  int tid = threadIdx.x;
  hold(tid);  // what follows from it is not kept for the next tile
  int bad = 0;  // 1: some value is not finite, 2: at a position that some row sees
#pragma unroll 1
  for (int i = tid; i < kChunks; i += kThreads) {
    const u32x4 w = v_lds[i];
    if (!(FP8 ? any_nonfinite_f16(w) : any_nonfinite_bf16(w))) continue;
    const int row = i / (kTile / 8), x = x0 + (((i % (kTile / 8)) ^ ((row >> 1) & 7)) * 8);  // of the chunk: v_chunk
    bad |= x + 8 > begin && x < end ? 3 : 1;
  }
  const int any = workgroup_bits(bad, sm.bits);
  if (any == 0) return;
  if (any & 2) {
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
        uint32_t* at = sm.marks + (row * (D / 32) + (d >> 5)) * 2;
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

// Row r of an item: its token in the sequence, and its query head.
struct LaneRow {
  bool live;
  int tok, hq;
};
__device__ __forceinline__ LaneRow lane_row(int r, int nrows, int group, int head) {
  LaneRow x;
  x.live = r < nrows;
  x.tok = x.live ? (int)((unsigned)r / (unsigned)group) : 0;
  x.hq = head * group + (x.live ? r - x.tok * group : 0);
  return x;
}

// Tiles t_begin .. t_stop - 1 of an item: its output (slot < 0: they are all of
// it), or a part of it into the workspace's slot.  True: nothing was written, it
// is to be done again, `careful` (LDS is free for it).
template <int D, bool FP8>
__device__ __forceinline__ bool attn_chunk_part(const tb_paged_attention_args& a, const AttnPlan& plan,
                                                const LineItem& it, int t_begin, int t_stop, int64_t slot, bool careful,
                                                const AttnShared& sm) {
  typedef ChunkOps<FP8> O;
  typedef typename O::Elem Elem;
  typedef typename O::V8 V8;
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
  // what follows from the thread is found again each time: kept for the next
  // part, it would cost registers that the loop over the tiles has not
  int own = threadIdx.x;
  hold(own);
  const int lane = own & 63, wave = uniform(own >> 6);
  const int i32 = lane & 31, half = lane >> 5;

  // the positions (low, pos] that the lane's row sees, and its wave's first and last row
  const LaneRow row = lane_row(r0 + wave * 32 + i32, nrows, group, head);
  const bool row_live = row.live;
  const int pos = s.first_pos + row.tok;
  auto behind_window = [&](int last) {
    return a.window > 0 && (int64_t)last - a.window > -1 ? (int)((int64_t)last - a.window) : -1;
  };
  const int low = behind_window(pos);
  const int w_first = r0 + wave * 32 < nrows ? r0 + wave * 32 : nrows - 1;
  const int w_last = w_first + 31 < nrows ? w_first + 31 : nrows - 1;
  const int pos_first = uniform(s.first_pos + (int)((unsigned)w_first / (unsigned)group));
  const int pos_last = uniform(s.first_pos + (int)((unsigned)w_last / (unsigned)group));
  // Tiles whose first position is in (w_low, w_high] are seen whole by all of
  // the wave's rows, those in (all_low, all_high] by all of the workgroup's
  // (none if values are taken out of every tile).
  const int w_low = behind_window(pos_last), w_high = pos_first - (kTile - 1);
  const int all_low = behind_window(s.first_pos + j_last);
  const int all_high = careful ? -__INT_MAX__ - 1 : s.first_pos + j_first - (kTile - 1);

  // scores are scaled by |scale|; its sign goes into the queries.  A scale of
  // 0 is taken as the smallest number, so that an unseen -inf stays one.
  float scale2 = a.scale * kLog2e * (FP8 && c.k_scale ? c.k_scale[head] : 1.f);
  const uint32_t flip = scale2 < 0.f ? 0x80008000u : 0u;
  scale2 = fmaxf(fabsf(scale2), 1.17549435e-38f);
  bf16x8 q[KK];
  {
    const uint16_t* qp =
        static_cast<const uint16_t*>(a.q) + (s.row0 + row.tok) * a.q_stride + (int64_t)row.hq * D + 8 * half;
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
  const uint32_t k_off = ((k_row & 15) * D + k_ch * kPer) * sizeof(Elem);  // bytes, inside a run
  const int v_off = v_row * c.page + (v_ch * kPer & 15);
  // An entry as it is loaded: paged_id of it, and so the wait for it, is left
  // for when it is needed (with the check here, a wave stood 1100 of a tile's
  // 5700 cycles waiting for the entry and all loads before it).
  auto lookup = [&](int t) -> int32_t {
    const int x = (first_tile + t) * kTile + 16 * v_run;
    int32_t entry = -1;
    if (t < t_end && (x | (c.page - 1)) >= span.begin && x < span.end) entry = paged_entry(table, c.table_width, x >> shift);
    return entry;
  };
  auto holder = [&](int g) { return FP8 ? g : 2 * g ^ 4 * (wave & 1); };  // bf16: row v_row of lanes 0..7 is 8 wave
  auto run_page = [&](int pages, int g) { return __builtin_amdgcn_readlane(pages, holder(g)); };
  u32x4 kr[FP8 ? kLoads : 1], vr[FP8 ? kLoads : 1];
  const int page_bytes = c.page * D * (int)sizeof(Elem);
  const int page_runs = c.page < kTile ? c.page / 16 : kTile / 16;  // runs of a tile that share a page
  const bool one_page = c.page >= kTile;                            // all of a tile's do
  auto page_of = [&](const Elem* cache, int page) { return cache + (page < 0 ? 0 : page) * page_step; };
  auto stage_k = [&](int t, int pages, u32x4* to) {
    const int x0 = (first_tile + t) * kTile;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int run = (i * kStep + uniform(k_row)) >> 4;
      const Elem* page = page_of(kc, run_page(pages, run));
      const int at = ((x0 + 16 * run) & (c.page - 1)) * D * (int)sizeof(Elem);
      if constexpr (FP8) kr[i] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(page) + at + k_off);
      else load_lds16(page, page_bytes, (int)k_off, at, &to[i * 64 * kWaves + wave * 64]);
    }
  };
  auto stage_v = [&](int t, int pages, u32x4* to) {
    const int x0 = (first_tile + t) * kTile;
    const int at = (x0 + 16 * v_run) & (c.page - 1);
    if constexpr (FP8) {
      const Elem* vp = page_of(vc, pages) + at + v_off;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) vr[i] = *reinterpret_cast<const u32x4*>(vp + i * vStep * c.page);
      return;
    }
    // A load is of one page: with several in a tile, of the lanes whose run lies in it.
    const int lane_at = (v_off + at) * (int)sizeof(Elem), step = vStep * c.page * (int)sizeof(Elem);
#pragma unroll 1
    for (int g = 0; g < kTile / 16; g += page_runs) {
      if (v_run < g || v_run >= g + page_runs) continue;
      const Elem* page = page_of(vc, run_page(pages, g));
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load_lds16(page, page_bytes, lane_at, i * step, &to[i * 64 * kWaves + wave * 64]);
    }
  };
  // The same for a tile within one page, one load at a time: `page` and `at` are
  // found once a tile.
  struct Loads {
    const Elem* page;
    int at;  // of the lane
  };
  auto loads_k = [&](int t, int pages) {
    const int slot = (((first_tile + t) * kTile) & (c.page - 1)) + (uniform(k_row) & ~15);
    return Loads{page_of(kc, run_page(pages, 0)), (int)k_off + slot * D * (int)sizeof(Elem)};
  };
  auto loads_v = [&](int t, int pages) {
    const int slot = ((first_tile + t) * kTile + 16 * v_run) & (c.page - 1);
    return Loads{page_of(vc, run_page(pages, 0)), (v_off + slot) * (int)sizeof(Elem)};
  };
  auto load_k = [&](const Loads& x, int i, u32x4* to) {
    load_lds16(x.page, page_bytes, x.at, i * kStep * D * (int)sizeof(Elem), &to[i * 64 * kWaves + wave * 64]);
  };
  auto load_v = [&](const Loads& x, int i, u32x4* to) {
    load_lds16(x.page, page_bytes, x.at, i * vStep * c.page * (int)sizeof(Elem), &to[i * 64 * kWaves + wave * 64]);
  };
  // 8-bit: the staged registers into LDS
  auto widen_k = [&](u32x4* to) {
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        to[k_chunk<D>(i * kStep + k_row, 2 * k_ch)] = __builtin_bit_cast(u32x4, fp8_to_bf16(u32x2{kr[i][0], kr[i][1]}));
        to[k_chunk<D>(i * kStep + k_row, 2 * k_ch + 1)] = __builtin_bit_cast(u32x4, fp8_to_bf16(u32x2{kr[i][2], kr[i][3]}));
      }
    }
  };
  auto widen_v = [&](u32x4* to) {
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        to[v_chunk(i * vStep + v_row, 2 * v_ch)] = __builtin_bit_cast(u32x4, fp8_to_f16(u32x2{vr[i][0], vr[i][1]}));
        to[v_chunk(i * vStep + v_row, 2 * v_ch + 1)] = __builtin_bit_cast(u32x4, fp8_to_f16(u32x2{vr[i][2], vr[i][3]}));
      }
    }
  };

  // matrix row m of a score tile stands for position key(m) of its 32: a
  // lane's score registers 0..7 are then positions 8 half + 0..7, 8..15 are 16 more
  const int key = 16 * (i32 >> 4) + 8 * ((i32 >> 2) & 1) + 4 * ((i32 >> 3) & 1) + (i32 & 3);

  // maximum (log2 units), and what the weights are relative to: its reference, or 0
  float m = -__builtin_inff(), base = 0.f;
  float l = 0.f;                            // the lane's sum
  f32x16 o[DT], sc[2];                      // scores of the first and of the second 32 positions of a tile
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[dt][e] = 0.f;
  float top = 0.f;  // of the lane's newest scores

  auto runs_of = [&](int pages) -> uint32_t {  // which of a tile's runs exist
    if (one_page) return run_page(pages, 0) < 0 ? 0u : 0xfu;
    uint32_t there = 0xfu;
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (run_page(pages, g) < 0) there &= ~(1u << g);
    return there;
  };

  // New scores (part u of tile t): what the rows do not see out, the maximum,
  // and the values' sums rescaled if it has grown by more than 2^kSlack.  Until
  // then weights stay relative to the older one: nothing is rounded more.
  auto settle = [&](f32x16& x, int t, int u, uint32_t there) {
    const int x0 = (first_tile + t) * kTile;
    if (!(there == 0xfu && x0 <= w_high && x0 > w_low)) {
      const int rel = x0 + 32 * u + 8 * half;  // positions have 30 bits
      const int hi = row_live ? (pos - rel < -1 ? -1 : pos - rel > 31 ? 31 : pos - rel) : -1;
      const int lo = low - rel < -1 ? -1 : low - rel > 31 ? 31 : low - rel;
      top = -__builtin_inff();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int y = 16 * (e >> 3) + (e & 7);
        const bool see = y <= hi && y > lo && ((there >> (2 * u + (e >> 3))) & 1u);
        x[e] = see ? x[e] : -__builtin_inff();
        top = fmaxf(top, x[e]);
      }
    }
    float t0, t1;
    swap_halves(top, t0, t1);
    const float row_top = fmaxf(t0, t1) * scale2;
    if (__ballot(row_top > m + (float)O::kSlack) != 0) {
      const float m_new = fmaxf(m, row_top);
      const float base_new = m_new == -__builtin_inff() ? 0.f : weight_reference<O::kRoom>(m_new);
      const float alpha = m == -__builtin_inff() ? 1.f : exp2_fast(base - base_new);
      m = m_new;
      base = base_new;
      l *= alpha;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[dt][e] *= alpha;
    }
  };

  // Scores `now` become weights and their values' sums (part uv of v_lds),
  // beside the products of the scores `next` (part uk of the keys in k_lds).
  // issue(i) is load i of a later tile: one every four products, as all at once
  // they stand in line.
  auto beside = [&](f32x16& now, f32x16& next, const u32x4* k_lds, int uk, const u32x4* v_lds, int uv, auto issue) {
    static_assert(2 * DT == KK, "as many products of values as of keys");
    constexpr int kProducts = 2 * KK, kAhead = 4;
    constexpr int kScores = 16 / KK;  // scores turned beside a product of keys
    u32x4 operand[kProducts];
    V8 w[2];
    auto load = [&](int i) {  // of product i: the keys' come first
      operand[i] = i < KK ? k_lds[k_chunk<D>(32 * uk + key, 2 * i + half)]
                          : v_lds[v_chunk(32 * ((i - KK) % DT) + i32, 2 * (2 * uv + (i - KK) / DT) + half)];
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i);
#pragma unroll
    for (int x = 0; x < 16; ++x) next[x] = 0.f;
    // Each round: an operand from LDS for a later product, a product, and what
    // the vector unit does meanwhile.  The compiler keeps the rounds as they
    // are; left to itself it forms the products in a row and then the weights.
#pragma unroll
    for (int i = 0; i < kProducts; ++i) {
      if (i + kAhead < kProducts) load(i + kAhead);
      if (i % 4 == 1) issue(i / 4);
      if (i < KK) {
        next = mfma32(__builtin_bit_cast(bf16x8, operand[i]), q[i], next);
#pragma unroll
        for (int k = 0; k < kScores; ++k) {
          const int x = i * kScores + k;
          const float p = exp2_fast(fmaf(now[x], scale2, -base));
          l += p;
          w[x >> 3][x & 7] = O::narrow(p);
        }
      } else {
        o[(i - KK) % DT] = mfma32(__builtin_bit_cast(V8, operand[i]), w[(i - KK) / DT], o[(i - KK) % DT]);
        if (i >= KK + KK / 2) {
          constexpr int kEach = 32 / KK;
#pragma unroll
          for (int k = 0; k < kEach; ++k) {
            const int x = (i - KK - KK / 2) * kEach + k;
            top = x == 0 ? next[0] : fmaxf(top, next[x]);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    hold(l);  // here, not where it is next used
    hold(top);
  };

  bool marked = false;
#pragma unroll
  for (int i = 0; i < kRows * D / 16 / (64 * kWaves); ++i) sm.marks[i * 64 * kWaves + tid] = 0u;  // a barrier follows
  const bool idle = r0 + wave * 32 >= nrows;  // the wave has no row: it only loads
  const int32_t e0 = lookup(t_begin), e1 = lookup(t_begin + 1), e2 = lookup(t_begin + 2);
  int p0 = paged_id(e0, c.n_pages), p1 = paged_id(e1, c.n_pages), p2 = paged_id(e2, c.n_pages);
  if (t_begin < t_end) {
    stage_k(t_begin, p0, sm.buffer[0]);
    stage_v(t_begin, p0, sm.buffer[2]);
    widen_k(sm.buffer[0]);
    widen_v(sm.buffer[2]);
    if (t_begin + 1 < t_end) {
      stage_k(t_begin + 1, p1, sm.buffer[1]);
      widen_k(sm.buffer[1]);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (!idle) {
#pragma unroll
      for (int x = 0; x < 16; ++x) sc[0][x] = sc[1][x] = 0.f;
#pragma unroll
      for (int i = 0; i < KK; ++i)
        sc[0] = mfma32(__builtin_bit_cast(bf16x8, sm.buffer[0][k_chunk<D>(key, 2 * i + half)]), q[i], sc[0]);
      top = sc[0][0];
#pragma unroll
      for (int x = 1; x < 16; ++x) top = fmaxf(top, sc[0][x]);
      settle(sc[0], t_begin, 0, runs_of(p0));
    }
  }
  // Tile t: K in k_lds, V in v_lds, K of t + 1 in k_next; V of t + 1 goes to
  // v_next, and K of t + 2, once all scores of t are formed, to k_lds.  The four
  // are arrays of their own, and which is which is known when this is compiled:
  // the compiler then knows that reading the one does not wait for the loads
  // into the other.
  auto step = [&](auto one, int t, u32x4* k_lds, u32x4* k_next, u32x4* v_lds, u32x4* v_next) {
    constexpr bool kOne = decltype(one)::value;  // bf16, in tiles within a page: loads go out beside the products
    static_assert(FP8 || 4 * kLoads == 2 * KK, "a load for four products");
    // V of t has come: what was issued after it (K of t + 1) may still be on its way
    if (!FP8 && t + 1 < t_end) wait_loads<kLoads>();
    else wait_loads<0>();
    __syncthreads();
    const int32_t e3 = lookup(t + 3);
    Loads ahead{};
    if constexpr (kOne) ahead = loads_v(t + 1, p1);
    else if (t + 1 < t_end) stage_v(t + 1, p1, v_next);
    auto ahead_v = [&](int i) {
      if constexpr (kOne) load_v(ahead, i, v_next);
    };
    const int x0 = (first_tile + t) * kTile;
    const uint32_t there = runs_of(p0);
    if (!(there == 0xfu && x0 <= all_high && x0 > all_low))
      take_nonfinite_tile<D, FP8, kRows>(v_lds, sm, marked, x0, there, span.begin, span.end, s.first_pos, group, r0, nrows,
                                         a.window);
    if (!idle) {
      beside(sc[0], sc[1], k_lds, 1, v_lds, 0, ahead_v);
      settle(sc[1], t, 1, there);
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) ahead_v(i);
    }
    wait_loads<FP8 ? 0 : kLoads>();  // K of t + 1 has come; V of t + 1, issued after it, may be on its way
    __syncthreads();
    const int p3 = paged_id(e3, c.n_pages);
    if constexpr (kOne) ahead = loads_k(t + 2, p2);
    else if (t + 2 < t_end) stage_k(t + 2, p2, k_lds);
    auto ahead_k = [&](int i) {
      if constexpr (kOne) load_k(ahead, i, k_lds);
    };
    if (!idle) {
      beside(sc[1], sc[0], k_next, 0, v_lds, 1, ahead_k);  // past the last tile: scores of what lies in k_next, not used
      if (t + 1 < t_end) settle(sc[0], t + 1, 0, runs_of(p1));
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) ahead_k(i);
    }
    widen_v(v_next);
    if (t + 2 < t_end) widen_k(k_lds);
    p0 = p1;
    p1 = p2;
    p2 = p3;
  };
  auto all = [&](auto one) {
    for (int t = t_begin; t < t_end; t += 2) {
      step(one, t, sm.buffer[0], sm.buffer[1], sm.buffer[2], sm.buffer[3]);
      if (t + 1 < t_end) step(one, t + 1, sm.buffer[1], sm.buffer[0], sm.buffer[3], sm.buffer[2]);
    }
  };
  if (!FP8 && one_page) {
    all(std::true_type());
    wait_loads<0>();  // past the last tile its loads were of the pool's first page, for nobody
  } else {
    all(std::false_type());
  }

  // the row's sum, and its output: register 4 j + e of tile dt is channel 32 dt + 8 j + 4 half + e
  {
    float a0, a1;
    swap_halves(l, a0, a1);
    l = a0 + a1;
  }
  // found again: kept through the loop, it would cost registers that the loop has not
  int thread = threadIdx.x;
  hold(thread);
  const int r = r0 + (thread >> 6) * 32 + (thread & 31), c0 = 4 * (thread >> 5 & 1);
  const LaneRow out = lane_row(r, nrows, group, head);
  if (!FP8 && !careful) {
    bool bad = false;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) bad = bad || any_nonfinite(o[dt], 16);
    bad = bad && out.live && fabsf(l) < __builtin_inff();  // else all of the row is NaN
    if (workgroup_bits(bad, sm.bits)) return true;
  }
  if (!out.live) return false;
  if (marked) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4 x = marked_sum<D>(sm.marks, r - r0, dt, 8 * j + c0);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[dt][4 * j + e] += x[e];
      }
  }
  const int64_t at = (s.row0 + out.tok) * a.heads_q + out.hq;
  const float ref = weight_reference<O::kRoom>(m);
  if (slot >= 0) {
    const int64_t pr = slot * kRows + (r - r0);
    if (c0 == 0) plan.chunk_line.stats[pr] = float2{ref, l};
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<f32x4*>(plan.chunk_line.values + pr * D + 32 * dt + 8 * j + c0) =
            f32x4{o[dt][4 * j], o[dt][4 * j + 1], o[dt][4 * j + 2], o[dt][4 * j + 3]};
    return false;
  }
  const RowScale rs = row_scale(a, head, at, c0 == 0, ref, l);
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      write4(a, at * D + 32 * dt + 8 * j + c0,
             f32x4{o[dt][4 * j], o[dt][4 * j + 1], o[dt][4 * j + 2], o[dt][4 * j + 3]}, rs);
  return false;
}

}  // namespace tb
