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
// The running maximum and sum of each row are kept in log2 units; sums and
// values are relative to weight_reference of the maximum, and what goes to LDS
// and to the workspace as the maximum is that reference.
//
// What bounds it: the cache's bytes.  Every K and V byte is loaded once,
// straight into operand registers (no LDS, no barrier in the loop), and each
// half of a tile's registers is loaded again, for the wave's next tile, as soon
// as its product is formed.  A token of each of 16 sequences of 2048..8192, 8
// key/value heads: 357 MB in 70.4 us, 5.1 TB/s; of 4 sequences of 16384..65536
// in e4m3: 330 MB in 63.2 us, 5.2 TB/s (a plain copy moves 5.1 TB/s).  One
// sequence of 1000 with 40 key/value heads: 10.4 us, of which 2 are to find the
// piece, 3 to the first tile, and 5 the launch and the joins of the waves.
//
// The four waves of a workgroup take the position tiles of a part in turn and
// join through LDS.
#pragma once

#include "attn_line.h"

namespace tb {

template <bool FP8>
struct RowOps;

template <>
struct RowOps<false> {
  typedef uint16_t Elem;
  static constexpr int kBlocks = 1;  // 32-position blocks per tile
  static constexpr int kRoom = 0;    // weights are at most 2^kRoom (weight_reference)
  typedef bf16x8 V8;
};

template <>
struct RowOps<true> {
  typedef uint8_t Elem;
  static constexpr int kBlocks = 2;
  static constexpr int kRoom = 15;  // 2^16 is past fp16's largest
  typedef f16x8 V8;
};

__device__ __forceinline__ f32x4 mfma16(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(const f16x8& a, const f16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Tiles t0 .. t1 - 1 of an item: its output (slot < 0: they are all of it), or
// a part of it into the workspace's slot.  True: nothing was written, it is to be
// done again, `careful` (values that are not finite are taken out of every tile).
template <int D, bool FP8>
__device__ __forceinline__ bool attn_rows_part(const tb_paged_attention_args& a, const AttnPlan& plan,
                                               const LineItem& it, int t0, int t1, int64_t slot, bool careful,
                                               const AttnShared& sm) {
  typedef RowOps<FP8> O;
  typedef typename O::Elem Elem;
  typedef typename O::V8 V8;
  constexpr int NB = O::kBlocks;          // 32-position blocks of a tile
  constexpr int T = rows_positions(FP8);  // positions of a tile
  constexpr int S = 2 * NB;               // 16-row score tiles of a tile
  constexpr int KL = D / 32 / NB;         // 16-byte loads of a key row per lane
  constexpr int DT = D / 16;              // 16-row tiles of O'

  const tb_paged_cache& c = a.cache;
  const int group = plan.group, head = it.head, nrows = it.seq.rows;  // one row tile: r is the row of the sequence
  const PagedSeq& s = it.seq.seq;
  const PagedSpan& span = it.span;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int i16 = lane & 15, q4 = lane >> 4;
  const int j1 = uniform((unsigned)(nrows - 1) / (unsigned)group);  // last token
  const int first_tile = it.held.first, t_end = t1 < it.held.count ? t1 : it.held.count;

  const int32_t* table = c.block_table + it.b * c.table_stride;
  const int shift = plan.shift, page = c.page;
  const int64_t page_step = (int64_t)c.heads_kv * page * D;
  const Elem* kc = static_cast<const Elem*>(c.k_cache) + (int64_t)head * page * D;
  const Elem* vc = static_cast<const Elem*>(c.v_cache) + (int64_t)head * page * D;

  // positions of the lane inside a tile: its key row (of score tile t, u):
  // krow + 8 t + 4 u, and its values: v0 .. v0 + 8 NB - 1
  const int krow = 8 * NB * (i16 >> 2) + (i16 & 3);
  const int v0 = 8 * NB * q4;

  // The table's entry for position x, -1 if nobody sees its page (it is not read
  // then).  paged_id of it, and so the wait for it, is left for when its tile is
  // loaded.
  auto entry_of = [&](int x) -> int32_t {
    int32_t entry = -1;
    if ((x | (page - 1)) >= span.begin && x < span.end) entry = paged_entry(table, c.table_width, x >> shift);
    return entry;
  };
  struct Pages {
    int32_t k, v;  // of the lane's keys and values
  };
  auto lookup = [&](int t) -> Pages {
    if (t >= t_end) return Pages{-1, -1};
    const int x0 = (first_tile + t) * T;
    return Pages{entry_of(x0 + krow), entry_of(x0 + v0)};
  };
  auto checked = [&](const Pages& p) { return Pages{paged_id(p.k, c.n_pages), paged_id(p.v, c.n_pages)}; };
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

  int t = t0 + wave;
  Tile ta;
  const Pages first = lookup(t);
  Pages ahead = lookup(t + kAttnWaves);

  // the lane's row
  const int r = i16;
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

  const Pages pa = checked(first);
  load_keys(ta, t, pa);
  load_values(ta, t, pa);

  float m = -__builtin_inff(), ref = m, l = 0.f;
  f32x4 o[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) o[dt] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Tile t, held in `x`, which is loaded again for the tile after the next.
  auto step = [&](Tile& x, int t) {
    const int x0 = (first_tile + t) * T, pv = x.page;
    // asked for before that tile's loads: loads return in order, and the next
    // step waits for this answer only
    const Pages now = checked(ahead);
    ahead = lookup(t + 2 * kAttnWaves);
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
    load_keys(x, t + kAttnWaves, now);

    // scores in log2 units; what the row does not see is -inf.  The lane's
    // scores and its values are of the same positions, so of one page.
#pragma unroll
    for (int st = 0; st < S; ++st)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[st][e] *= scale2;
    // every row of the tile sees every position of it
    const bool full = !careful && __ballot(pv < 0) == 0 && x0 + T - 1 <= s.first_pos &&
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
    const float ref_new = weight_reference<O::kRoom>(m_new);
    const float base = m_new == -__builtin_inff() ? 0.f : ref_new;
    const float alpha = m == -__builtin_inff() ? 1.f : keep_infinity(exp2_fast(ref - base));
    m = m_new;
    ref = ref_new;
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
    load_values(x, t + kAttnWaves, now);
  };
  while (t < t_end) {
    step(ta, t);
    t += kAttnWaves;
  }

  constexpr int kRow = D + 4;  // floats of a row in LDS
  // the waves' sums joined: each scales its values to the common maximum
  l = sum_over_rows(l);
  if (q4 == 0) {
    sm.max[wave * 16 + i16] = ref;
    sm.sum[wave * 16 + i16] = l;
  }
  if constexpr (!FP8) {
    bool bad = false;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) bad = bad || any_nonfinite(o[dt], 4);
    // a sum that is not finite makes all of the row NaN
    sm.bits[wave] = !careful && __ballot(bad && row_live && fabsf(l) < __builtin_inff()) != 0 ? 1 : 0;
  }
  __syncthreads();
  if constexpr (!FP8) {
    int any = 0;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) any |= sm.bits[w];
    if (uniform(any) != 0) {
      __syncthreads();
      return true;
    }
  }
  {
    float top = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) top = fmaxf(top, sm.max[w * 16 + i16]);
    const float f = keep_infinity(exp2_fast(ref - (top == -__builtin_inff() ? 0.f : top)));
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      if (w != wave) continue;
      f32x4* to = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(sm.buffer[w]) + i16 * kRow + 4 * q4);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) to[4 * dt] = o[dt] * f;
    }
  }
  __syncthreads();
  constexpr int DL = D / 16;  // channels of a thread: 16 threads a row
  const int d0 = (threadIdx.x & 15) * DL, row = threadIdx.x >> 4;
  if (row >= nrows) return false;
  float top = -__builtin_inff(), total = 0.f;
#pragma unroll
  for (int w = 0; w < kAttnWaves; ++w) top = fmaxf(top, sm.max[w * 16 + row]);
  const float base = top == -__builtin_inff() ? 0.f : top;
  f32x4 v[DL / 4];
#pragma unroll
  for (int e = 0; e < DL / 4; ++e) v[e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < kAttnWaves; ++w) {
    total = fmaf(sm.sum[w * 16 + row], exp2_fast(sm.max[w * 16 + row] - base), total);
#pragma unroll
    for (int e = 0; e < DL / 4; ++e)
      v[e] += *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(sm.buffer[w]) + row * kRow + d0 + 4 * e);
  }
  if (slot >= 0) {
    const int64_t pr = slot * kRowsTile + row;
    if (d0 == 0) plan.rows_line.stats[pr] = float2{top, total};
#pragma unroll
    for (int e = 0; e < DL / 4; ++e) *reinterpret_cast<f32x4*>(plan.rows_line.values + pr * D + d0 + 4 * e) = v[e];
    return false;
  }
  const int otok = (unsigned)row / (unsigned)group;
  const int64_t at = (s.row0 + otok) * a.heads_q + head * group + (row - otok * group);
  const RowScale rs = row_scale(a, head, at, d0 == 0, top, total);
#pragma unroll
  for (int e = 0; e < DL / 4; ++e) write4(a, at * D + d0 + 4 * e, v[e], rs);
  return false;
}

}  // namespace tb
