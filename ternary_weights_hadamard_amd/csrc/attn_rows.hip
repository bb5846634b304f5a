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
// straight into operand registers (no LDS, no barrier in the loop); the next
// tile's keys and this tile's values are in flight while scores are formed.
// The four waves of a workgroup take tiles in turn and join at the end through
// LDS; positions are also split over workgroups until the GPU is full, and the
// parts are joined by a second launch.
#include "attn_common.h"
#include "attn_launch.h"

namespace tb {

namespace {

constexpr int kWaves = 4;

template <bool FP8>
struct Ops;

template <>
struct Ops<false> {
  typedef uint16_t Elem;
  static constexpr int kBlocks = 1;  // 32-position blocks per tile
  typedef bf16x8 V8;
};

template <>
struct Ops<true> {
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

template <int D, bool FP8>
__global__ void __launch_bounds__(64 * kWaves, 2) attn_rows_kernel(tb_paged_attention_args a, AttnPlan plan,
                                                                  int row_tiles) {
  typedef Ops<FP8> O;
  typedef typename O::Elem Elem;
  typedef typename O::V8 V8;
  constexpr int NB = O::kBlocks;      // 32-position blocks of a tile
  constexpr int T = rows_positions(FP8);  // positions of a tile
  constexpr int S = 2 * NB;           // 16-row score tiles of a tile
  constexpr int KL = D / 32 / NB;     // 16-byte loads of a key row per lane
  constexpr int DT = D / 16;          // 16-row tiles of O'
  __shared__ float sm_max[kWaves][16], sm_sum[kWaves][16];
  __shared__ __align__(16) float sm_o[kWaves][16][D + 4];

  const tb_paged_cache& c = a.cache;
  const int64_t b = blockIdx.z;
  const int group = a.heads_q / c.heads_kv;
  const int64_t width = c.n_pages > 0 ? c.table_width : 0;
  const PagedSeq s = paged_seq(c.cu_q, c.kv_len, b, c.total_q, width * c.page);
  const int64_t n = s.n < c.max_q ? s.n : c.max_q;
  const int64_t nrows = n * group;
  // Consecutive workgroups go to the eight dies in turn; the row tiles of one
  // (part, head) read the same positions, so they are eight apart.
  const int eighth = blockIdx.x & 7, rest = blockIdx.x >> 3;
  const int rt = rest % row_tiles, pair = rest / row_tiles * 8 + eighth;
  const int head = pair % c.heads_kv, split = pair / c.heads_kv;
  const int64_t r0 = (int64_t)rt * kRowsTile;
  if (r0 >= nrows || split >= plan.by_rows.splits || plan.is_chunk(nrows)) return;
  const int64_t rl = r0 + kRowsTile - 1 < nrows ? r0 + kRowsTile - 1 : nrows - 1;  // last row
  const PagedSpan span = paged_span(s, (int)(r0 / group), (int)(rl / group), a.window);
  const TileSpan all = tile_span(span, T);
  const int parts = plan.by_rows.parts(all.count), first_tile = all.first;
  if (split >= parts) return;
  const int t_begin = split * plan.by_rows.tiles;
  const int t_end = split + 1 == parts ? all.count : t_begin + plan.by_rows.tiles;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i16 = lane & 15, q4 = lane >> 4;

  // the lane's row
  const int64_t r = r0 + i16;
  const bool row_live = r < nrows;
  const int tok = row_live ? (int)(r / group) : 0;
  const int hq = head * group + (row_live ? (int)(r % group) : 0);
  const int64_t pos = (int64_t)s.first_pos + tok;               // sees positions <= pos ..
  const int64_t low = a.window > 0 ? pos - a.window : -1;       // .. and > low
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

  const int32_t* table = c.block_table + b * c.table_stride;
  const int shift = __builtin_ctz(c.page);
  const Elem* kc = static_cast<const Elem*>(c.k_cache);
  const Elem* vc = static_cast<const Elem*>(c.v_cache);
  const int64_t page_elems = (int64_t)c.page * D;

  // positions of the lane inside a tile: its key row (of score tile t, u):
  // krow + 8 t + 4 u, and its values: v0 .. v0 + 8 NB - 1
  const int krow = 8 * NB * (i16 >> 2) + (i16 & 3);
  const int v0 = 8 * NB * q4;

  // The page of position x, or -1 (none, or nobody sees it; its table entry is not read then).
  auto page_of = [&](int64_t x) -> int {
    if ((x | (c.page - 1)) < span.begin || x >= span.end) return -1;
    return paged_page(table, c.table_width, c.n_pages, x >> shift);
  };

  float m = -__builtin_inff(), l = 0.f;
  f32x4 o[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) o[dt] = f32x4{0.f, 0.f, 0.f, 0.f};

  u32x4 kr[S][KL];
  auto load_keys = [&](int t, int page) {
    const int64_t x0 = (int64_t)(first_tile + t) * T;
    const Elem* p = kc + ((int64_t)(page < 0 ? 0 : page) * c.heads_kv + head) * page_elems;
#pragma unroll
    for (int st = 0; st < S; ++st) {
      const int x = krow + 8 * (st >> 1) + 4 * (st & 1);
      const Elem* row = p + (int64_t)((x0 + x) & (c.page - 1)) * D + (16 / sizeof(Elem)) * q4;
#pragma unroll
      for (int kk = 0; kk < KL; ++kk) kr[st][kk] = *reinterpret_cast<const u32x4*>(row + 32 * NB * kk);
    }
  };

  int t = t_begin + wave;
  int pk = -1, pv = -1;  // pages of the lane's keys and values
  if (t < t_end) {
    const int64_t x0 = (int64_t)(first_tile + t) * T;
    pk = page_of(x0 + krow);
    pv = page_of(x0 + v0);
    load_keys(t, pk);
  }
  while (t < t_end) {
    const int64_t x0 = (int64_t)(first_tile + t) * T;
    const int tn = t + kWaves;
    // the next tile's pages, then this tile's values
    int pk_next = -1, pv_next = -1;
    if (tn < t_end) {
      const int64_t xn = (int64_t)(first_tile + tn) * T;
      pk_next = page_of(xn + krow);
      pv_next = page_of(xn + v0);
    }
    u32x4 vr[DT];
    {
      const Elem* p = vc + ((int64_t)(pv < 0 ? 0 : pv) * c.heads_kv + head) * page_elems + ((x0 + v0) & (c.page - 1));
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) vr[dt] = *reinterpret_cast<const u32x4*>(p + (int64_t)(16 * dt + i16) * c.page);
    }

    f32x4 sc[S];
#pragma unroll
    for (int st = 0; st < S; ++st) {
      sc[st] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < KL; ++kk) {
        if constexpr (FP8) {
          const u32x4 w = kr[st][kk];
          sc[st] = mfma16(fp8_to_bf16(u32x2{w[0], w[1]}), q[2 * kk], sc[st]);
          sc[st] = mfma16(fp8_to_bf16(u32x2{w[2], w[3]}), q[2 * kk + 1], sc[st]);
        } else {
          sc[st] = mfma16(__builtin_bit_cast(bf16x8, kr[st][kk]), q[kk], sc[st]);
        }
      }
    }
    if (tn < t_end) load_keys(tn, pk_next);

    // scores in log2 units; what the row does not see is -inf.  The lane's
    // scores and its values are of the same positions, so of one page.
#pragma unroll
    for (int st = 0; st < S; ++st)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[st][e] *= scale2;
    // every row of the tile sees every position of it
    const bool full = __ballot(pv < 0) == 0 && x0 + T - 1 <= (int64_t)s.first_pos + r0 / group &&
                      (a.window <= 0 || x0 > (int64_t)s.first_pos + rl / group - a.window);
    uint32_t seen = 0xffffffffu;  // bit 4 st + e
    if (!full) {
      seen = 0;
#pragma unroll
      for (int st = 0; st < S; ++st)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t x = x0 + v0 + 8 * (st >> 1) + 4 * (st & 1) + e;
          const bool see = row_live && pv >= 0 && x <= pos && x > low;
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
      for (int dt = 0; dt < DT; ++dt) bad = bad || (FP8 ? any_nonfinite_fp8(vr[dt]) : any_nonfinite_bf16(vr[dt]));
      if (__ballot(bad) != 0) {
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          f32x4 up = {0.f, 0.f, 0.f, 0.f}, down = up;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            V8 v, see;
#pragma unroll
            for (int e = 0; e < 8; ++e) see[e] = (seen >> (8 * nb + e)) & 1u ? 1.f : 0.f;
            if constexpr (FP8) v = fp8_to_f16(u32x2{vr[dt][2 * nb], vr[dt][2 * nb + 1]});
            else v = __builtin_bit_cast(bf16x8, vr[dt]);
            const Nonfinite<V8> nf = take_nonfinite(v);
            up = mfma16(nf.up, see, up);
            down = mfma16(nf.down, see, down);
            if constexpr (!FP8) vr[dt] = __builtin_bit_cast(u32x4, v);
          }
          if constexpr (FP8) vr[dt] = drop_nonfinite_fp8(vr[dt]);
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
          o[dt] = mfma16(fp8_to_f16(u32x2{vr[dt][2 * nb], vr[dt][2 * nb + 1]}), w, o[dt]);
        } else {
          const bf16x8 v = __builtin_bit_cast(bf16x8, vr[dt]);
          o[dt] = mfma16(v, w, o[dt]);
          o[dt] = mfma16(v, low_w, o[dt]);
        }
      }
    }
    pv = pv_next;
    t = tn;
  }

  // the waves' sums joined: each scales its values to the common maximum
  l = sum_over_rows(l);
  if (q4 == 0) {
    sm_max[wave][i16] = m;
    sm_sum[wave][i16] = l;
  }
  __syncthreads();
  {
    float top = sm_max[0][i16];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, sm_max[w][i16]);
    const float f = exp2_fast(m - (top == -__builtin_inff() ? 0.f : top));
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) *reinterpret_cast<f32x4*>(&sm_o[wave][i16][16 * dt + 4 * q4]) = o[dt] * f;
  }
  __syncthreads();
  constexpr int DL = D / 16;  // channels of a thread: 16 threads a row
  const int orow = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * DL;
  if (r0 + orow >= nrows) return;
  float top = sm_max[0][orow], total = 0.f;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) top = fmaxf(top, sm_max[w][orow]);
  const float base = top == -__builtin_inff() ? 0.f : top;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) total = fmaf(sm_sum[w][orow], exp2_fast(sm_max[w][orow] - base), total);
  float v[DL];
#pragma unroll
  for (int e = 0; e < DL; ++e) {
    v[e] = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v[e] += sm_o[w][orow][d0 + e];
  }
  const int64_t at = (s.row0 + (r0 + orow) / group) * a.heads_q + head * group + (r0 + orow) % group;
  if (parts > 1) {
    const int64_t pr = (int64_t)split * plan.rows + at;
    if (d0 == 0) plan.stats[pr] = float2{top, total};
    if (total == 0.f) return;
#pragma unroll
    for (int e = 0; e < DL; e += 4)
      *reinterpret_cast<f32x4*>(plan.values + pr * D + d0 + e) = f32x4{v[e], v[e + 1], v[e + 2], v[e + 3]};
    return;
  }
  const RowScale rs = row_scale(a, head, at, d0 == 0, top, total);
#pragma unroll
  for (int e = 0; e < DL; e += 4) write4(a, at * D + d0 + e, f32x4{v[e], v[e + 1], v[e + 2], v[e + 3]}, rs);
}

}  // namespace

hipError_t launch_attn_rows(const tb_paged_attention_args& a, const AttnPlan& plan, hipStream_t stream) {
  const tb_paged_cache& c = a.cache;
  int64_t rows = c.max_q * (a.heads_q / c.heads_kv);
  if (rows > plan.few) rows = plan.few;
  const int row_tiles = (int)((rows + kRowsTile - 1) / kRowsTile);
  const int64_t pairs = (int64_t)c.heads_kv * plan.by_rows.splits;
  const dim3 grid((unsigned)((pairs + 7) / 8 * 8 * row_tiles), 1, (unsigned)c.B), block(64 * kWaves);
  const bool f8 = c.cache_dtype == TB_FP8;
  if (c.head_dim == 64) {
    if (f8) hipLaunchKernelGGL((attn_rows_kernel<64, true>), grid, block, 0, stream, a, plan, row_tiles);
    else hipLaunchKernelGGL((attn_rows_kernel<64, false>), grid, block, 0, stream, a, plan, row_tiles);
  } else {
    if (f8) hipLaunchKernelGGL((attn_rows_kernel<128, true>), grid, block, 0, stream, a, plan, row_tiles);
    else hipLaunchKernelGGL((attn_rows_kernel<128, false>), grid, block, 0, stream, a, plan, row_tiles);
  }
  return hipGetLastError();
}

}  // namespace tb
