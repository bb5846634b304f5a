// tb_paged_attention: its kernels, how a call is cut, and its launches.
#include "attn_chunk.h"
#include "tb_launch.h"

namespace tb {

namespace {

// The first plan.chunk_blocks workgroups are for chunks, the others for few
// rows.  Batches of one kind launch its kernel alone; both kinds together use
// no more registers or LDS than the chunks do.
template <int D, bool FP8, bool ROWS, bool CHUNK>
__global__ void __launch_bounds__(64 * kAttnWaves, 2) attn_kernel(tb_paged_attention_args a, AttnPlan plan) {
  constexpr int kBuffer = CHUNK ? kChunkPositions * D * 2 : kRowsTile * (D + 4) * 4;  // bytes
  static_assert(kBuffer >= kRowsTile * (D + 4) * 4, "both kinds share the buffers");
  __shared__ u32x4 b0[kBuffer / 16], b1[kBuffer / 16], b2[kBuffer / 16], b3[kBuffer / 16];
  __shared__ float stats[2][16 * kAttnWaves];
  __shared__ int bits[kAttnWaves];
  __shared__ uint32_t marks[CHUNK ? kChunkTile * D / 16 : 1];
  const AttnShared sm{{b0, b1, b2, b3}, stats[0], stats[1], bits, marks};
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (CHUNK && (!ROWS || block < plan.chunk_blocks)) {
    if constexpr (CHUNK)
      run_line<true, FP8>(a, plan, block, [&](const LineItem& it, int t0, int t1, int64_t slot, bool careful) {
        return attn_chunk_part<D, FP8>(a, plan, it, t0, t1, slot, careful, sm);
      });
  } else if constexpr (ROWS) {
    run_line<false, FP8>(a, plan, block - plan.chunk_blocks, [&](const LineItem& it, int t0, int t1, int64_t slot, bool careful) {
      return attn_rows_part<D, FP8>(a, plan, it, t0, t1, slot, careful, sm);
    });
  }
}

// The parts of row r's item: of a sequence of the kind, one head.
template <bool CHUNK, bool FP8>
__device__ __forceinline__ LineParts parts_of_row(const tb_paged_attention_args& a, const AttnPlan& plan, int64_t b,
                                                  const LineSeq& seq, int head, int r) {
  typedef LineKind<CHUNK, FP8> K;
  const AttnLine& cut = CHUNK ? plan.chunk_line : plan.rows_line;
  const int rt = (unsigned)r / (unsigned)K::kRows;
  const int tiles = K::tiles(a, plan, seq, rt);
  Line<CHUNK, FP8> line(a, plan);
  int64_t start = line.before(a, plan, b);
  if constexpr (CHUNK) start += a.cache.heads_kv * K::tiles_before(a, plan, seq, rt);
  return line_parts(start + (int64_t)head * tiles, tiles, cut.piece(line.total));
}

// Row r in `parts`, joined by L = 16 lanes (a wave does four) or by all 64
// (rows in many parts: what counts is the time of one).  Lane p of them holds the
// statistics of part p, of L at a time, and their groups of 16 take the parts
// in turn, D / 16 channels a lane.  Bound by latency: the line again, a row's
// statistics and its first parts (16 rows of 40 heads 6.1 us; 8 x 45 rows of 8
// key/value heads in 8 parts each 8.4 us by whole waves, 14.5 us by 16 lanes).
template <int D, bool CHUNK, bool FP8, int L>
__device__ __forceinline__ void join_row(const tb_paged_attention_args& a, const AttnPlan& plan, const LineParts& parts,
                                         const LineSeq& seq, int head, int r) {
  constexpr int kRows = LineKind<CHUNK, FP8>::kRows, G = L / 16;
  constexpr int DL = D / 16, kBatch = 4;  // parts whose loads a lane has in flight
  const AttnLine& cut = CHUNK ? plan.chunk_line : plan.rows_line;
  const int lane = threadIdx.x & (L - 1), g = lane >> 4, d0 = (lane & 15) * DL;
  const int64_t row = (unsigned)r % (unsigned)kRows;

  float top = -__builtin_inff(), total = 0.f;
  f32x4 v[DL / 4];
#pragma unroll
  for (int e = 0; e < DL / 4; ++e) v[e] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int c0 = 0; c0 < parts.count; c0 += L) {
    float2 st = {-__builtin_inff(), 0.f};
    if (c0 + lane < parts.count) st = cut.stats[parts.slot(c0 + lane) * kRows + row];
    float base = 0.f, f = 0.f;
    for (int p0 = c0; p0 < parts.count && p0 < c0 + L; p0 += G * kBatch) {
      f32x4 x[kBatch][DL / 4];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int p = p0 + G * u + g < parts.count ? p0 + G * u + g : parts.count - 1;  // past the last: weight 0
        const float* from = cut.values + (parts.slot(p) * kRows + row) * D + d0;
#pragma unroll
        for (int e = 0; e < DL / 4; ++e) x[u][e] = *reinterpret_cast<const f32x4*>(from + 4 * e);
      }
      if (p0 == c0) {  // the statistics of these parts, behind the first loads
        float t = st.x;
#pragma unroll
        for (int m = 1; m < L; m <<= 1) t = fmaxf(t, __shfl_xor(t, m));
        const float now = fmaxf(top, t);
        base = now == -__builtin_inff() ? 0.f : now;
        f = exp2_fast(st.x - base);
        const float alpha = exp2_fast(top - base);
        top = now;
        total = fmaf(total, alpha, st.y * f);
#pragma unroll
        for (int e = 0; e < DL / 4; ++e) v[e] *= keep_infinity(alpha);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int p = p0 + G * u + g;
        const float w = keep_infinity(__shfl(f, p - c0, L));
#pragma unroll
        for (int e = 0; e < DL / 4; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (p < parts.count) v[e][i] = fmaf(x[u][e][i], w, v[e][i]);
      }
    }
  }
#pragma unroll
  for (int m = 1; m < 16; m <<= 1) total += __shfl_xor(total, m);
  if constexpr (G > 1) {
    total = sum_over_rows(total);
#pragma unroll
    for (int e = 0; e < DL / 4; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[e][i] = sum_over_rows(v[e][i]);
    if (g != 0) return;
  }
  const int tok = (unsigned)r / (unsigned)plan.group;
  const int64_t at = (seq.seq.row0 + tok) * a.heads_q + head * plan.group + (r - tok * plan.group);
  const RowScale rs = row_scale(a, head, at, d0 == 0, top, total);
#pragma unroll
  for (int e = 0; e < DL / 4; ++e) write4(a, at * D + d0 + 4 * e, v[e], rs);
}

// ROWS (16, or 4 by whole waves) rows of one key/value head of one sequence.
template <int D, bool FP8, int ROWS>
__global__ void __launch_bounds__(256) attn_join_kernel(tb_paged_attention_args a, AttnPlan plan) {
  const unsigned heads = (unsigned)a.cache.heads_kv;
  const int head = blockIdx.x % heads, r0 = blockIdx.x / heads * ROWS;
  const int64_t b = blockIdx.z;
  const LineSeq chunk = LineKind<true, FP8>::sequence(a, plan, b), few = LineKind<false, FP8>::sequence(a, plan, b);
  if (plan.chunk_line.pieces && r0 < chunk.rows) {  // all of one row tile
    const LineParts parts = parts_of_row<true, FP8>(a, plan, b, chunk, head, r0);
    const int r = r0 + (int)(ROWS == 16 ? threadIdx.x >> 4 : uniform(threadIdx.x >> 6));
    if (parts.count > 1 && r < chunk.rows) join_row<D, true, FP8, ROWS == 16 ? 16 : 64>(a, plan, parts, chunk, head, r);
  }
  if (plan.rows_line.pieces && r0 < few.rows) {
    const LineParts parts = parts_of_row<false, FP8>(a, plan, b, few, head, r0);
    if (parts.count == 1) return;  // written by its kernel
    for (int r = r0 + uniform(threadIdx.x >> 6); r < r0 + ROWS && r < few.rows; r += 4)
      join_row<D, false, FP8, 64>(a, plan, parts, few, head, r);
  }
}

constexpr int kPieces = 512;  // two workgroups for each of 256 CUs

// rows of the largest sequence
int64_t most_rows(const tb_paged_attention_args& a) {
  return most_tokens(a.cache.max_q, a.cache.total_q) * (a.heads_q / a.cache.heads_kv);
}

// Whether sequences may have more rows than `few`, and whether any may go to the
// kernel for few rows.  Token arrays of exactly B times the most tokens are most
// likely those of B equal sequences; as the lengths are not known here, the
// chunk kernel, launched alone, then takes the short ones too (few is 0).
bool has_chunk(const tb_paged_attention_args& a, const AttnPlan& p) { return most_rows(a) > p.few; }
bool has_rows(const tb_paged_attention_args& a, const AttnPlan& p) {
  return !has_chunk(a, p) || a.cache.total_q != a.cache.B * most_tokens(a.cache.max_q, a.cache.total_q);
}

// the items of chunks, at most
int64_t chunk_items(const tb_paged_attention_args& a, const AttnPlan& p) {
  return most_row_tiles(a.cache.total_q, a.cache.B, p.group, p.few, kChunkTile) * a.cache.heads_kv;
}

AttnPlan plan_of(const tb_paged_attention_args& a) {
  const tb_paged_cache& c = a.cache;
  AttnPlan p{};
  p.few = kRowsTile;
  if (!has_rows(a, p)) p.few = 0;
  p.capacity = c.n_pages > 0 ? c.table_width * c.page : 0;
  p.group = a.heads_q / c.heads_kv;
  p.shift = __builtin_ctz(c.page);
  int64_t keys = a.window > 0 && a.window + c.max_q < a.max_kv ? a.window + c.max_q : a.max_kv;
  if (keys > TB_MAX_POSITIONS) keys = TB_MAX_POSITIONS;
  p.rows_line.least = 8;
  p.rows_line.slot_rows = kRowsTile;
  p.chunk_line.least = 4;
  p.chunk_line.slot_rows = kChunkTile;
  if (has_rows(a, p) && keys > p.rows_line.least * rows_positions(c.cache_dtype == TB_FP8)) p.rows_line.pieces = kPieces;
  // Chunks whose items fill the GPU are not cut: one after another, the row
  // tiles of a head find its keys and values in L2, while pieces of a line are
  // all elsewhere (4 x 2048 tokens over 8192, 40 heads, an earlier form of the
  // kernel: 625 us as items, 883 us as pieces).  Nor are those of fewer items if it saves less than ten tiles,
  // which is what a second part's start, the parts' way through memory and the
  // join take, and pieces run two on a CU, where each takes 5/4 of its time (2 x
  // 777 tokens of 16 heads: 18 tiles within a window of 1000 38.6 us as items,
  // 36 + 12 as pieces; 94 tiles without one 141 and 95 + 12).
  const int64_t seen = a.window + (kChunkTile - 1) / p.group + 1;  // by a row tile, in a window
  const int64_t most = a.window > 0 && seen < keys ? seen : keys;
  const int64_t tiles = (most + kChunkPositions - 1) / kChunkPositions, items = chunk_items(a, p);
  if (has_chunk(a, p) && items < kPieces && tiles - tiles * items * 5 / (4 * kPieces) > 10) p.chunk_line.pieces = kPieces;
  return p;
}

// bytes of a line's values (a multiple of 16), and of its statistics
size_t value_bytes(const tb_paged_attention_args& a, const AttnLine& l) {
  return 2 * (size_t)l.pieces * (size_t)l.slot_rows * (size_t)a.cache.head_dim * sizeof(float);
}
size_t stat_bytes(const AttnLine& l) { return 2 * (size_t)l.pieces * (size_t)l.slot_rows * sizeof(float2); }

template <int D, bool FP8>
hipError_t launch(const tb_paged_attention_args& a, AttnPlan p, hipStream_t stream) {
  const tb_paged_cache& c = a.cache;
  const bool chunk = has_chunk(a, p), rows = has_rows(a, p);
  p.chunk_blocks = !chunk ? 0 : p.chunk_line.pieces ? p.chunk_line.pieces : chunk_items(a, p);
  const int64_t few = !rows ? 0 : p.rows_line.pieces ? p.rows_line.pieces : c.B * c.heads_kv;
  const GridXY xy = grid_of(p.chunk_blocks + few);
  const dim3 grid(xy.x, xy.y), block(64 * kAttnWaves);
  if (!chunk) hipLaunchKernelGGL((attn_kernel<D, FP8, true, false>), grid, block, 0, stream, a, p);
  else if (!rows) hipLaunchKernelGGL((attn_kernel<D, FP8, false, true>), grid, block, 0, stream, a, p);
  else hipLaunchKernelGGL((attn_kernel<D, FP8, true, true>), grid, block, 0, stream, a, p);
  const hipError_t e = hipGetLastError();
  const int64_t few_rows = !p.rows_line.pieces ? 0 : most_rows(a) < p.few ? most_rows(a) : p.few;
  const int64_t joined = p.chunk_line.pieces ? most_rows(a) : few_rows;
  if (e != hipSuccess || joined == 0) return e;
  // Rows of many chunk items are in few parts each, and are many.
  const bool many = p.chunk_line.pieces && chunk_items(a, p) > kPieces / 4;
  const int each = many ? 16 : 4;
  const dim3 join((unsigned)((joined + each - 1) / each * c.heads_kv), 1, (unsigned)c.B);
  if (many) hipLaunchKernelGGL((attn_join_kernel<D, FP8, 16>), join, dim3(256), 0, stream, a, p);
  else hipLaunchKernelGGL((attn_join_kernel<D, FP8, 4>), join, dim3(256), 0, stream, a, p);
  return hipGetLastError();
}

}  // namespace

size_t attn_part_bytes(const tb_paged_attention_args& a) {
  const AttnPlan p = plan_of(a);
  return value_bytes(a, p.rows_line) + stat_bytes(p.rows_line) + value_bytes(a, p.chunk_line) + stat_bytes(p.chunk_line);
}

hipError_t launch_paged_attention(const tb_paged_attention_args& a, bool split, hipStream_t stream) {
  AttnPlan p = plan_of(a);
  char* w = static_cast<char*>(a.workspace);
  for (AttnLine* l : {&p.rows_line, &p.chunk_line}) {
    if (!split) l->pieces = 0;
    l->values = reinterpret_cast<float*>(w);
    w += value_bytes(a, *l);
    l->stats = reinterpret_cast<float2*>(w);
    w += stat_bytes(*l);
  }
  const bool f8 = a.cache.cache_dtype == TB_FP8;
  if (a.cache.head_dim == 64) return f8 ? launch<64, true>(a, p, stream) : launch<64, false>(a, p, stream);
  return f8 ? launch<128, true>(a, p, stream) : launch<128, false>(a, p, stream);
}

}  // namespace tb
