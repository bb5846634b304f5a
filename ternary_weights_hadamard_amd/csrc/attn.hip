// How a tb_paged_attention call is split, its launches, and the kernel that
// joins the parts of split positions.
#include "attn_chunk.h"
#include "tb_launch.h"

namespace tb {

namespace {

constexpr int kMaxParts = 64;  // of a chunk's row tile

// The first plan.chunk_blocks * B workgroups are for chunks, the others for few
// rows.  Batches of one kind launch its kernel alone; both kinds together use
// no more registers or LDS than the chunks do.
template <int D, bool FP8, bool ROWS, bool CHUNK>
__global__ void __launch_bounds__(64 * kAttnWaves, 2) attn_kernel(tb_paged_attention_args a, AttnPlan plan) {
  union Shared {
    RowsShared<D> rows;
    ChunkShared<D> chunk;
  };
  __shared__ __align__(16) unsigned char shared[CHUNK ? sizeof(Shared) : sizeof(RowsShared<D>)];
  unsigned block = blockIdx.x;
  if constexpr (CHUNK) {
    const unsigned chunks = plan.chunk_blocks * (unsigned)a.cache.B;
    if (!ROWS || block < chunks) {
      attn_chunk<D, FP8>(a, plan, block % plan.chunk_blocks, block / plan.chunk_blocks,
                         *reinterpret_cast<ChunkShared<D>*>(shared));
      return;
    }
    block -= chunks;
  }
  if constexpr (ROWS) {
    RowsShared<D>& sm = *reinterpret_cast<RowsShared<D>*>(shared);
    if (plan.pieces) attn_rows<D, FP8>(a, plan, block, sm);
    else attn_rows_whole<D, FP8>(a, plan, block, sm);
  }
}

// 16 lanes a row, D / 16 channels each.  Few rows: the parts of an item, in the
// slots of the pieces it lies in.
template <int D>
__device__ __forceinline__ void join_rows(const tb_paged_attention_args& a, const AttnPlan& plan, int64_t b, int head,
                                          int r, const RowsSeq& seq) {
  constexpr int DL = D / 16;
  const int64_t before = rows_before(a, plan, b), total = rows_total(a, plan), per = plan.piece(total);
  if (r >= seq.rows) return;
  const int tiles = line_tiles(seq);
  const int64_t start = before + (int64_t)head * tiles;
  const int64_t w0 = start / per, w1 = (start + tiles - 1) / per;
  if (w0 == w1) return;  // one part: written by its kernel
  const int i16 = threadIdx.x & 15, d0 = i16 * DL, parts = (int)(w1 - w0 + 1);
  // piece w0 ends with this item, unless it starts with it; the others start with it
  const int64_t slot0 = 2 * w0 + (w0 * per < start ? 1 : 0);
  auto row_of = [&](int p) -> int64_t { return (p == 0 ? slot0 : 2 * (w0 + p)) * plan.slot_rows + r; };
  float top = -__builtin_inff();
  for (int p = i16; p < parts; p += 16) top = fmaxf(top, plan.rows_stats[row_of(p)].x);
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
  const float base = top == -__builtin_inff() ? 0.f : top;
  float total_w = 0.f;
  f32x4 v[DL / 4];
#pragma unroll
  for (int e = 0; e < DL / 4; ++e) v[e] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int p0 = 0; p0 < parts; p0 += 4) {
    // four parts' loads at once; past the last part the weight is 0
    f32x4 x[4][DL / 4];
    float2 st[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t pr = row_of(p0 + u < parts ? p0 + u : parts - 1);
      st[u] = plan.rows_stats[pr];
#pragma unroll
      for (int e = 0; e < DL / 4; ++e) x[u][e] = *reinterpret_cast<const f32x4*>(plan.rows_values + pr * D + d0 + 4 * e);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float f = p0 + u < parts ? exp2_fast(st[u].x - base) : 0.f;
      if (p0 + u < parts) total_w = fmaf(st[u].y, f, total_w);
#pragma unroll
      for (int e = 0; e < DL / 4; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (p0 + u < parts) v[e][i] = fmaf(x[u][e][i], f, v[e][i]);
    }
  }
  const int tok = (unsigned)r / (unsigned)plan.group;
  const int64_t at = (seq.seq.row0 + tok) * a.heads_q + head * plan.group + (r - tok * plan.group);
  const RowScale rs = row_scale(a, head, at, i16 == 0, top, total_w);
#pragma unroll
  for (int e = 0; e < DL / 4; ++e) write4(a, at * D + d0 + 4 * e, v[e], rs);
}

// Chunks: each lane holds the statistics of every 16th part.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(tb_paged_attention_args a, AttnPlan plan) {
  constexpr int DL = D / 16, kHeld = kMaxParts / 16;
  const tb_paged_cache& c = a.cache;
  const int64_t b = blockIdx.z;
  const int head = blockIdx.x % (unsigned)c.heads_kv, rt = blockIdx.x / (unsigned)c.heads_kv;
  const int group = plan.group;
  const PagedSeq s = paged_seq(c.cu_q, c.kv_len, b, c.total_q, plan.capacity);
  const int nrows = (s.n < (int)c.max_q ? s.n : (int)c.max_q) * group;
  const int r = rt * 16 + (int)(threadIdx.x >> 4);
  if (!plan.is_chunk(nrows)) {
    if (plan.pieces && rt * 16 < nrows) join_rows<D>(a, plan, b, head, r, rows_seq(a, plan, b));
    return;
  }
  if (r >= nrows) return;
  // the parts of the row's tile, as its kernel cut them
  const int r0 = r / kChunkTile * kChunkTile;
  const int rl = r0 + kChunkTile - 1 < nrows ? r0 + kChunkTile - 1 : nrows - 1;
  const PagedSpan span =
      paged_span(s, (unsigned)r0 / (unsigned)group, (unsigned)rl / (unsigned)group, a.window);
  const int parts = plan.by_chunk.parts(tile_span(span, kChunkPositions).count);
  if (parts == 1) return;  // written by its kernel
  const int i16 = threadIdx.x & 15, d0 = i16 * DL;
  const int tok = (unsigned)r / (unsigned)group;
  const int64_t at = (s.row0 + tok) * a.heads_q + head * group + (r - tok * group);

  float2 st[kHeld];
  float top = -__builtin_inff();
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int p = 16 * k + i16;
    st[k] = float2{-__builtin_inff(), 0.f};
    if (p < parts) st[k] = plan.stats[p * plan.rows + at];
  }
#pragma unroll
  for (int k = 0; k < kHeld; ++k) top = fmaxf(top, st[k].x);
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
  const float base = top == -__builtin_inff() ? 0.f : top;
  float total = 0.f, f[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    f[k] = st[k].y == 0.f ? 0.f : exp2_fast(st[k].x - base);
    total += st[k].y * f[k];
  }
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) total += __shfl_xor(total, x);

  f32x4 v[DL / 4];
#pragma unroll
  for (int e = 0; e < DL / 4; ++e) v[e] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float* values = plan.values + at * D + d0;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int here = parts - 16 * k < 16 ? parts - 16 * k : 16;
    for (int p0 = 0; p0 < here; p0 += 4) {
      // four parts' loads at once; past the last part the weight is 0
      f32x4 x[4][DL / 4];
      float w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int p = 16 * k + p0 + u < parts ? 16 * k + p0 + u : parts - 1;
        w[u] = __shfl(f[k], p0 + u, 16);
#pragma unroll
        for (int e = 0; e < DL / 4; ++e)
          x[u][e] = *reinterpret_cast<const f32x4*>(values + p * plan.rows * D + 4 * e);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < DL / 4; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i)  // a part without weight holds no values: what is read there counts as 0
            v[e][i] = fmaf(w[u] == 0.f ? 0.f : x[u][e][i], w[u], v[e][i]);
    }
  }
  const RowScale rs = row_scale(a, head, at, i16 == 0, top, total);
#pragma unroll
  for (int e = 0; e < DL / 4; ++e) write4(a, at * D + d0 + 4 * e, v[e], rs);
}

// Parts of the `keys` positions that bring `items` workgroups to about `want`:
// at least `least` tiles each, at most kMaxParts of them.
AttnSplit split_to(int64_t items, int64_t want, int64_t keys, int positions, int least) {
  const int64_t all = (keys + positions - 1) / positions;
  int64_t tiles = (items * all + want - 1) / want;
  if (tiles < least) tiles = least;
  if (tiles < (all + kMaxParts - 1) / kMaxParts) tiles = (all + kMaxParts - 1) / kMaxParts;
  const int64_t parts = (all + tiles - 1) / tiles;
  return AttnSplit{(int)(parts < 1 ? 1 : parts), (int)tiles};
}

// rows of the largest sequence
int64_t most_rows(const tb_paged_attention_args& a) { return a.cache.max_q * (a.heads_q / a.cache.heads_kv); }

constexpr int kPieces = 512;  // two workgroups for each of 256 CUs

// The bytes of the workspace's arrays, each a multiple of 16.
struct Parts {
  size_t values, stats, rows_values, rows_stats;
  size_t all() const { return values + stats + rows_values + rows_stats; }
};

AttnPlan plan_of(const tb_paged_attention_args& a) {
  const tb_paged_cache& c = a.cache;
  AttnPlan p{};
  p.few = 64;
  p.rows = c.total_q * a.heads_q;
  p.capacity = c.n_pages > 0 ? c.table_width * c.page : 0;
  p.group = a.heads_q / c.heads_kv;
  p.shift = __builtin_ctz(c.page);
  const int64_t most = most_rows(a), few = most < p.few ? most : p.few;
  int64_t keys = a.window > 0 && a.window + c.max_q < a.max_kv ? a.window + c.max_q : a.max_kv;
  if (keys > TB_MAX_POSITIONS) keys = TB_MAX_POSITIONS;
  const bool chunk = most > p.few, rows = !chunk || c.total_q < c.B * c.max_q;  // all alike: chunks only
  p.least = 8;
  p.slot_rows = (int)((few + kRowsTile - 1) / kRowsTile * kRowsTile);
  // short items that fill the GPU by themselves are not cut
  const int64_t tiles = (keys + rows_positions(c.cache_dtype == TB_FP8) - 1) / rows_positions(c.cache_dtype == TB_FP8);
  p.pieces = rows && tiles > p.least ? kPieces : 0;
  p.by_chunk = AttnSplit{1, 1 << 30};
  if (chunk) {
    p.by_chunk = split_to((most + kChunkTile - 1) / kChunkTile * c.heads_kv * c.B, 1024, keys, kChunkPositions, 8);
    p.chunk_blocks = (unsigned)((most + kChunkTile - 1) / kChunkTile * c.heads_kv * p.by_chunk.splits);
  }
  return p;
}

Parts parts_of(const tb_paged_attention_args& a, const AttnPlan& p) {
  Parts s{};
  if (p.by_chunk.splits > 1) {
    const size_t n = (size_t)p.by_chunk.splits * (size_t)p.rows;
    s.values = n * a.cache.head_dim * 4;
    s.stats = (n * 8 + 15) / 16 * 16;
  }
  if (p.pieces) {
    const size_t n = 2 * (size_t)p.pieces * (size_t)p.slot_rows;
    s.rows_values = n * a.cache.head_dim * 4;
    s.rows_stats = n * 8;
  }
  return s;
}

template <int D, bool FP8>
hipError_t launch(const tb_paged_attention_args& a, const AttnPlan& p, hipStream_t stream) {
  const tb_paged_cache& c = a.cache;
  const int64_t most = most_rows(a);
  const bool chunk = most > p.few, rows = !chunk || c.total_q < c.B * c.max_q;
  const unsigned chunks = p.chunk_blocks * (unsigned)c.B;
  const unsigned few = rows ? (p.pieces ? (unsigned)p.pieces : (unsigned)(c.B * c.heads_kv)) : 0;
  const dim3 grid(chunks + few), block(64 * kAttnWaves);
  if (!chunk) hipLaunchKernelGGL((attn_kernel<D, FP8, true, false>), grid, block, 0, stream, a, p);
  else if (!rows) hipLaunchKernelGGL((attn_kernel<D, FP8, false, true>), grid, block, 0, stream, a, p);
  else hipLaunchKernelGGL((attn_kernel<D, FP8, true, true>), grid, block, 0, stream, a, p);
  const hipError_t e = hipGetLastError();
  // what may be in parts: nothing, the sequences with few rows, or any
  const int64_t joined = p.by_chunk.splits > 1 ? most : p.pieces ? (most < p.few ? most : p.few) : 0;
  if (e != hipSuccess || joined == 0) return e;
  hipLaunchKernelGGL((attn_join_kernel<D>), dim3((unsigned)((joined + 15) / 16 * c.heads_kv), 1, (unsigned)c.B), dim3(256),
                     0, stream, a, p);
  return hipGetLastError();
}

}  // namespace

size_t attn_part_bytes(const tb_paged_attention_args& a) { return parts_of(a, plan_of(a)).all(); }

hipError_t launch_paged_attention(const tb_paged_attention_args& a, bool split, hipStream_t stream) {
  const tb_paged_cache& c = a.cache;
  AttnPlan p = plan_of(a);
  if (!split) {
    p.by_chunk = AttnSplit{1, 1 << 30};
    if (p.chunk_blocks) p.chunk_blocks = (unsigned)((most_rows(a) + kChunkTile - 1) / kChunkTile * c.heads_kv);
    p.pieces = 0;
  } else {
    const Parts s = parts_of(a, p);
    char* w = static_cast<char*>(a.workspace);
    p.values = reinterpret_cast<float*>(w);
    p.stats = reinterpret_cast<float2*>(w + s.values);
    p.rows_values = reinterpret_cast<float*>(w + s.values + s.stats);
    p.rows_stats = reinterpret_cast<float2*>(w + s.values + s.stats + s.rows_values);
  }
  const bool f8 = c.cache_dtype == TB_FP8;
  if (c.head_dim == 64) return f8 ? launch<64, true>(a, p, stream) : launch<64, false>(a, p, stream);
  return f8 ? launch<128, true>(a, p, stream) : launch<128, false>(a, p, stream);
}

}  // namespace tb
