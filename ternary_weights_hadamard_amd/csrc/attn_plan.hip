// How a tb_paged_attention call is split, its launches, and the kernel that
// joins the parts of split positions.
#include "attn_launch.h"
#include "tb_launch.h"

namespace tb {

namespace {

// 16 lanes a row: each takes D / 16 channels of every part.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(tb_paged_attention_args a, AttnPlan plan) {
  constexpr int DL = D / 16;
  const tb_paged_cache& c = a.cache;
  const int64_t b = blockIdx.z;
  const int head = blockIdx.x % (unsigned)c.heads_kv, rt = blockIdx.x / (unsigned)c.heads_kv;
  const int group = a.heads_q / c.heads_kv;
  const int64_t width = c.n_pages > 0 ? c.table_width : 0;
  const PagedSeq s = paged_seq(c.cu_q, c.kv_len, b, c.total_q, width * c.page);
  const int64_t n = s.n < c.max_q ? s.n : c.max_q, nrows = n * group;
  const int64_t r = (int64_t)rt * 16 + (threadIdx.x >> 4);
  if (r >= nrows) return;
  // the parts of the row's tile, as its kernel cut them
  const bool chunk = plan.is_chunk(nrows);
  const int64_t size = chunk ? kChunkTile : kRowsTile, r0 = r / size * size;
  const int64_t rl = r0 + size - 1 < nrows ? r0 + size - 1 : nrows - 1;
  const PagedSpan span = paged_span(s, (int)(r0 / group), (int)(rl / group), a.window);
  const TileSpan all = tile_span(span, chunk ? kChunkPositions : rows_positions(c.cache_dtype == TB_FP8));
  const int splits = (chunk ? plan.by_chunk : plan.by_rows).parts(all.count);
  if (splits == 1) return;  // written by its kernel
  const int d0 = (threadIdx.x & 15) * DL;
  const int64_t at = (s.row0 + r / group) * a.heads_q + head * group + r % group;
  float top = -__builtin_inff();
  for (int p = 0; p < splits; ++p) top = fmaxf(top, plan.stats[p * plan.rows + at].x);
  const float base = top == -__builtin_inff() ? 0.f : top;
  float total = 0.f, v[DL];
#pragma unroll
  for (int e = 0; e < DL; ++e) v[e] = 0.f;
  for (int p = 0; p < splits; ++p) {
    const int64_t pr = p * plan.rows + at;
    const float2 st = plan.stats[pr];
    if (st.y == 0.f) continue;
    const float f = exp2_fast(st.x - base);
    total = fmaf(st.y, f, total);
#pragma unroll
    for (int e = 0; e < DL; e += 4) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(plan.values + pr * D + d0 + e);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[e + k] = fmaf(x[k], f, v[e + k]);
    }
  }
  const RowScale rs = row_scale(a, head, at, d0 == 0, top, total);
#pragma unroll
  for (int e = 0; e < DL; e += 4) write4(a, at * D + d0 + e, f32x4{v[e], v[e + 1], v[e + 2], v[e + 3]}, rs);
}

// Parts of the `keys` positions that bring `items` workgroups to about `want`:
// at least `least` tiles each, at most 64 of them.
AttnSplit split_to(int64_t items, int64_t want, int64_t keys, int positions, int least) {
  const int64_t all = (keys + positions - 1) / positions;
  int64_t tiles = (items * all + want - 1) / want;
  if (tiles < least) tiles = least;
  if (tiles < (all + 63) / 64) tiles = (all + 63) / 64;
  const int64_t parts = (all + tiles - 1) / tiles;
  return AttnSplit{(int)(parts < 1 ? 1 : parts), (int)tiles};
}

AttnPlan plan_of(const tb_paged_attention_args& a) {
  const tb_paged_cache& c = a.cache;
  AttnPlan p{};
  p.few = 32;
  p.rows = c.total_q * a.heads_q;
  const int64_t most = c.max_q * (a.heads_q / c.heads_kv);
  int64_t keys = a.window > 0 && a.window + c.max_q < a.max_kv ? a.window + c.max_q : a.max_kv;
  if (keys > TB_MAX_POSITIONS) keys = TB_MAX_POSITIONS;
  const int64_t few = most < p.few ? most : p.few;
  p.by_rows = split_to((few + kRowsTile - 1) / kRowsTile * c.heads_kv * c.B, 1024, keys,
                       rows_positions(c.cache_dtype == TB_FP8), 8);
  p.by_chunk = AttnSplit{1, 1 << 30};
  if (most > p.few)
    p.by_chunk = split_to((most + kChunkTile - 1) / kChunkTile * c.heads_kv * c.B, 1024, keys, kChunkPositions, 8);
  return p;
}

}  // namespace

int attn_splits(const tb_paged_attention_args& a) {
  const AttnPlan p = plan_of(a);
  return p.by_rows.splits > p.by_chunk.splits ? p.by_rows.splits : p.by_chunk.splits;
}

size_t attn_part_bytes(const tb_paged_attention_args& a, int splits) {
  if (splits <= 1) return 0;
  return (size_t)splits * (size_t)a.cache.total_q * (size_t)a.heads_q * ((size_t)a.cache.head_dim + 2) * sizeof(float);
}

hipError_t launch_paged_attention(const tb_paged_attention_args& a, int splits, hipStream_t stream) {
  const tb_paged_cache& c = a.cache;
  AttnPlan p = plan_of(a);
  if (splits == 1) {
    p.by_rows.splits = p.by_chunk.splits = 1;
  } else {
    p.values = static_cast<float*>(a.workspace);
    p.stats = reinterpret_cast<float2*>(p.values + (int64_t)splits * p.rows * c.head_dim);
  }
  const int64_t most = c.max_q * (a.heads_q / c.heads_kv);
  hipError_t e = hipSuccess;
  if (most > p.few) e = launch_attn_chunk(a, p, stream);
  // sequences with few rows among those: none if all have max_q tokens
  if (e == hipSuccess && (most <= p.few || c.total_q < c.B * c.max_q)) e = launch_attn_rows(a, p, stream);
  if (e != hipSuccess || splits == 1) return e;
  const unsigned items = (unsigned)((most + 15) / 16 * c.heads_kv);
  const dim3 grid(items, 1, (unsigned)c.B);
  if (c.head_dim == 64) hipLaunchKernelGGL((attn_join_kernel<64>), grid, dim3(256), 0, stream, a, p);
  else hipLaunchKernelGGL((attn_join_kernel<128>), grid, dim3(256), 0, stream, a, p);
  return hipGetLastError();
}

}  // namespace tb
