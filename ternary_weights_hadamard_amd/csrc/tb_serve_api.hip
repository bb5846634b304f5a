// C ABI of the serving operators: host-side argument validation, then their
// launches on the caller's stream.  Validation makes no HIP call.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tb.h"
#include "tb_check.h"
#include "tb_launch.h"

using namespace tb;

namespace {

// a byte range of the caller's
struct Range {
  const void* p;
  size_t bytes;
};

template <int N>
bool overlaps_any(const Range& a, const Range (&others)[N]) {
  for (const Range& o : others)
    if (overlap(a.p, a.bytes, o.p, o.bytes)) return true;
  return false;
}

// bytes from the first to past the last element of `rows` rows, `stride` elements apart
size_t strided_bytes(int64_t rows, int64_t stride, int64_t cols, size_t elem) {
  return rows <= 0 ? 0 : ((size_t)(rows - 1) * (size_t)stride + (size_t)cols) * elem;
}

int64_t norm_parts(const tb_block_norm_args& a) { return a.parts <= 1 ? 1 : a.parts; }

tb_status check_norm(const tb_block_norm_args& a) {
  if (!dtype_ok(a.h_dtype) || !dtype_ok(a.w_dtype) || !dtype_ok(a.gate_dtype) ||
      !(dtype_ok(a.z_dtype) || a.z_dtype == TB_ACT8) || !dtype_ok(a.y_dtype))
    return TB_ERR_DTYPE;
  if (a.parts > 1 && a.y_dtype != TB_F32) return TB_ERR_DTYPE;
  if (a.rows < 0 || a.rows > ((int64_t)1 << 35) || a.C <= 0 || a.C % 128 || a.C > TB_NORM_MAX_C || a.parts < 0 || a.parts > TB_MAX_PARTS)
    return TB_ERR_SHAPE;
  if (a.gate && a.rows_per_gate < 1) return TB_ERR_SHAPE;
  if (!isfinite(a.alpha) || !isfinite(a.eps) || !(a.eps > 0.f)) return TB_ERR_VALUE;
  if (a.rows == 0) return TB_OK;
  if (!a.h && !a.z) return TB_ERR_NULL;
  if (!a.y && !a.resid) return TB_ERR_NULL;
  if (a.z && !a.w_pre) return TB_ERR_NULL;
  const void* all[] = {a.y, a.resid, a.w_post, a.w_pre, a.gate, a.h, a.z};
  for (const void* p : all)
    if (!aligned16(p)) return TB_ERR_ALIGN;
  const size_t n = (size_t)a.rows * (size_t)a.C;
  const Range y{a.y, (size_t)norm_parts(a) * n * dtype_bytes(a.y_dtype)}, resid{a.resid, n * dtype_bytes(a.h_dtype)};
  const Range wq{a.w_post, (size_t)a.C * dtype_bytes(a.w_dtype)}, wp{a.w_pre, (size_t)a.C * dtype_bytes(a.w_dtype)};
  const int64_t gates = a.gate ? (a.rows - 1) / a.rows_per_gate + 1 : 0;
  const Range gate{a.gate, (size_t)gates * (size_t)a.C * dtype_bytes(a.gate_dtype)};
  const Range h{a.h, n * dtype_bytes(a.h_dtype)};
  const Range z{a.z, a.z_dtype == TB_ACT8 ? act8_bytes(n) : n * dtype_bytes(a.z_dtype)};
  const Range ins[] = {y, wq, wp, gate};
  if (overlaps_any(h, ins) || overlaps_any(z, ins) || overlap(h.p, h.bytes, z.p, z.bytes)) return TB_ERR_ALIAS;
  if (a.h != a.resid && overlap(h.p, h.bytes, resid.p, resid.bytes)) return TB_ERR_ALIAS;
  if (overlap(z.p, z.bytes, resid.p, resid.bytes)) return TB_ERR_ALIAS;
  return TB_OK;
}

// the cache and its metadata, without null pointers (those only when there is work)
tb_status check_cache_sizes(const tb_paged_cache& c) {
  if (c.cache_dtype != TB_BF16 && c.cache_dtype != TB_FP8) return TB_ERR_DTYPE;
  if (c.head_dim != 64 && c.head_dim != 128) return TB_ERR_SHAPE;
  if (c.page < 16 || c.page > TB_MAX_PAGE || (c.page & (c.page - 1))) return TB_ERR_SHAPE;
  if (c.B < 0 || c.B > 65535 || c.heads_kv < 1 || c.heads_kv > 65535 || c.n_pages < 0 || c.n_pages > INT32_MAX)
    return TB_ERR_SHAPE;
  if (c.total_q < 0 || c.total_q > TB_MAX_TOKENS || c.max_q < 0 || c.max_q > TB_MAX_TOKENS) return TB_ERR_SHAPE;
  if (c.table_width < 0 || c.table_stride < c.table_width) return TB_ERR_SHAPE;
  if (c.table_width > TB_MAX_POSITIONS / c.page) return TB_ERR_SHAPE;
  return TB_OK;
}

size_t cache_bytes(const tb_paged_cache& c) {
  return (size_t)c.n_pages * c.heads_kv * c.page * c.head_dim * (c.cache_dtype == TB_FP8 ? 1 : 2);
}

tb_status check_cache_pointers(const tb_paged_cache& c) {
  if (!c.cu_q || !c.kv_len) return TB_ERR_NULL;
  if (c.n_pages > 0 && (!c.k_cache || !c.v_cache)) return TB_ERR_NULL;
  if (c.table_width > 0 && !c.block_table) return TB_ERR_NULL;
  if (!aligned16(c.k_cache) || !aligned16(c.v_cache)) return TB_ERR_ALIGN;
  if (!aligned4(c.cu_q) || !aligned4(c.kv_len) || !aligned4(c.block_table) || !aligned4(c.k_scale) ||
      !aligned4(c.v_scale))
    return TB_ERR_ALIGN;
  return TB_OK;
}

bool stride_ok(int64_t stride, int64_t cols) {
  return stride >= cols && stride % 8 == 0 && stride <= ((int64_t)1 << 31);
}

tb_status check_attention_sizes(const tb_paged_attention_args& a) {
  const tb_paged_cache& c = a.cache;
  const tb_status st = check_cache_sizes(c);
  if (st != TB_OK) return st;
  if (!dtype_ok(a.out_dtype)) return TB_ERR_DTYPE;
  if (a.heads_q < 1 || a.heads_q > 65535 || a.heads_q % c.heads_kv) return TB_ERR_SHAPE;
  if (c.max_q * a.heads_q > TB_MAX_ROWS) return TB_ERR_SHAPE;
  if (a.window < 0 || a.window > INT32_MAX || a.max_kv < 0 || a.reserved != 0) return TB_ERR_SHAPE;
  if (!stride_ok(a.q_stride, (int64_t)a.heads_q * c.head_dim)) return TB_ERR_SHAPE;
  if (!isfinite(a.scale)) return TB_ERR_VALUE;
  return TB_OK;
}

}  // namespace

extern "C" {

tb_status tb_block_norm(const tb_block_norm_args* args, void* stream) {
  if (!args) return TB_ERR_NULL;
  const tb_status st = check_norm(*args);
  if (st != TB_OK || args->rows == 0) return st;
  tb_block_norm_args a = *args;
  a.parts = (int)norm_parts(a);
  return launched(launch_block_norm(a, as_stream(stream)));
}

tb_status tb_paged_append(const tb_paged_cache* cache, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, void* stream) {
  if (!cache) return TB_ERR_NULL;
  const tb_paged_cache& c = *cache;
  tb_status st = check_cache_sizes(c);
  if (st != TB_OK) return st;
  const int64_t row = (int64_t)c.heads_kv * c.head_dim;
  if (!stride_ok(k_stride, row) || !stride_ok(v_stride, row)) return TB_ERR_SHAPE;
  if (c.B == 0 || c.total_q == 0 || c.max_q == 0 || c.n_pages == 0 || c.table_width == 0) return TB_OK;
  st = check_cache_pointers(c);
  if (st != TB_OK) return st;
  if (!k || !v) return TB_ERR_NULL;
  if (!aligned16(k) || !aligned16(v)) return TB_ERR_ALIGN;
  const size_t cb = cache_bytes(c);
  const Range ins[] = {{k, strided_bytes(c.total_q, k_stride, row, 2)},
                       {v, strided_bytes(c.total_q, v_stride, row, 2)},
                       {c.cu_q, (size_t)(c.B + 1) * 4},
                       {c.kv_len, (size_t)c.B * 4},
                       {c.block_table, strided_bytes(c.B, c.table_stride, c.table_width, 4)},
                       {c.k_scale, (size_t)c.heads_kv * 4},
                       {c.v_scale, (size_t)c.heads_kv * 4}};
  if (overlaps_any({c.k_cache, cb}, ins) || overlaps_any({c.v_cache, cb}, ins) ||
      overlap(c.k_cache, cb, c.v_cache, cb))
    return TB_ERR_ALIAS;
  return launched(launch_paged_append(c, static_cast<const uint16_t*>(k), k_stride, static_cast<const uint16_t*>(v),
                                      v_stride, as_stream(stream)));
}

size_t tb_paged_attention_workspace(const tb_paged_attention_args* args) {
  if (!args || check_attention_sizes(*args) != TB_OK) return 0;
  const tb_paged_cache& c = args->cache;
  if (c.B == 0 || c.total_q == 0 || c.max_q == 0) return 0;
  return attn_part_bytes(*args);
}

tb_status tb_paged_attention(const tb_paged_attention_args* args, void* stream) {
  if (!args) return TB_ERR_NULL;
  const tb_paged_attention_args& a = *args;
  const tb_paged_cache& c = a.cache;
  tb_status st = check_attention_sizes(a);
  if (st != TB_OK || c.B == 0 || c.total_q == 0 || c.max_q == 0) return st;
  st = check_cache_pointers(c);
  if (st != TB_OK) return st;
  if (!a.q || !a.out) return TB_ERR_NULL;
  if (!aligned16(a.q) || !aligned16(a.out) || !aligned16(a.workspace) || !aligned4(a.lse)) return TB_ERR_ALIGN;
  const size_t need = attn_part_bytes(a);
  const bool split = need > 0 && a.workspace && a.workspace_bytes >= need;
  const size_t cb = cache_bytes(c), rows = (size_t)c.total_q * (size_t)a.heads_q;
  const Range out{a.out, rows * c.head_dim * dtype_bytes(a.out_dtype)}, lse{a.lse, rows * 4};
  const Range ws{a.workspace, split ? need : 0};
  const Range ins[] = {{c.k_cache, cb},
                       {c.v_cache, cb},
                       {a.q, strided_bytes(c.total_q, a.q_stride, (int64_t)a.heads_q * c.head_dim, 2)},
                       {c.cu_q, (size_t)(c.B + 1) * 4},
                       {c.kv_len, (size_t)c.B * 4},
                       {c.block_table, strided_bytes(c.B, c.table_stride, c.table_width, 4)},
                       {c.k_scale, (size_t)c.heads_kv * 4},
                       {c.v_scale, (size_t)c.heads_kv * 4}};
  if (overlaps_any(out, ins) || overlaps_any(lse, ins) || overlaps_any(ws, ins) ||
      overlap(out.p, out.bytes, lse.p, lse.bytes) || overlap(ws.p, ws.bytes, out.p, out.bytes) ||
      overlap(ws.p, ws.bytes, lse.p, lse.bytes))
    return TB_ERR_ALIAS;
  return launched(launch_paged_attention(a, split, as_stream(stream)));
}

size_t tb_verify_draft_workspace(int64_t B, int64_t vocab) {
  if (B <= 0 || B > 65535 || vocab <= kVerifyWhole || vocab > INT32_MAX) return 0;
  // two sums a slice, one count a sequence
  return ((size_t)B * (size_t)((vocab + kVerifySlice - 1) / kVerifySlice) * 16 + (size_t)B * 4 + 15) / 16 * 16;
}

tb_status tb_verify_draft(const tb_verify_draft_args* args, void* stream) {
  if (!args) return TB_ERR_NULL;
  const tb_verify_draft_args& a = *args;
  if (!dtype_ok(a.p_dtype) || !dtype_ok(a.q_dtype)) return TB_ERR_DTYPE;
  if (a.B < 0 || a.B > 65535 || a.total < 0 || a.total > TB_MAX_TOKENS || a.vocab <= 0 || a.vocab > INT32_MAX ||
      a.max_draft < 0 || a.max_draft > TB_MAX_DRAFT || a.reserved != 0)
    return TB_ERR_SHAPE;
  if (a.p_stride < a.vocab || a.p_stride > ((int64_t)1 << 32)) return TB_ERR_SHAPE;
  if (a.q && (a.q_stride < a.vocab || a.q_stride > ((int64_t)1 << 32))) return TB_ERR_SHAPE;
  if (a.B == 0) return TB_OK;
  if (!a.p || !a.u_next || !a.cu_draft || !a.accepted || !a.tokens) return TB_ERR_NULL;
  if (a.total > 0 && (!a.drafts || !a.u)) return TB_ERR_NULL;
  const size_t pe = dtype_bytes(a.p_dtype), qe = dtype_bytes(a.q_dtype);
  if (reinterpret_cast<uintptr_t>(a.p) % pe || reinterpret_cast<uintptr_t>(a.q) % qe || !aligned4(a.drafts) ||
      !aligned4(a.u) || !aligned4(a.u_next) || !aligned4(a.cu_draft) || !aligned4(a.accepted) || !aligned4(a.tokens) ||
      !aligned16(a.workspace))
    return TB_ERR_ALIGN;
  const size_t need = tb_verify_draft_workspace(a.B, a.vocab);
  if (need > 0 && (!a.workspace || a.workspace_bytes < need)) return TB_ERR_WORKSPACE;
  const Range ins[] = {{a.p, strided_bytes(a.total + a.B, a.p_stride, a.vocab, pe)},
                       {a.q, strided_bytes(a.total, a.q_stride, a.vocab, qe)},
                       {a.drafts, (size_t)a.total * 4},
                       {a.u, (size_t)a.total * 4},
                       {a.u_next, (size_t)a.B * 4},
                       {a.cu_draft, (size_t)(a.B + 1) * 4}};
  const Range outs[] = {{a.accepted, (size_t)a.B * 4},
                        {a.tokens, (size_t)a.B * (size_t)(a.max_draft + 1) * 4},
                        {a.workspace, need}};
  for (int i = 0; i < 3; ++i) {
    if (overlaps_any(outs[i], ins)) return TB_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return TB_ERR_ALIAS;
  }
  return launched(launch_verify_draft(a, as_stream(stream)));
}

}  // extern "C"
