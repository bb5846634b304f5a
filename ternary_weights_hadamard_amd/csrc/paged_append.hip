// New keys and values into the paged cache (include/tb.h, tb_paged_append).
//
// K pages are [position][d], so a token's row is copied as it is.  V pages are
// [d][position] (the attention loads 8 or 16 positions of one d as a matrix
// operand), so values are turned: a workgroup takes 64 positions of one head,
// holds their values in LDS as the cache's type, and writes each d's run of
// positions in 16-byte pieces where all of a piece is new.
#include "paged.h"
#include "tb_common.h"
#include "tb_launch.h"

namespace tb {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;  // positions per workgroup

// nearest e4m3 of x (ties to even), at most 448 in magnitude; NaN stays NaN
__device__ __forceinline__ uint32_t fp8_pair(float a, float b) {
  a = a > 448.f ? 448.f : a < -448.f ? -448.f : a;
  b = b > 448.f ? 448.f : b < -448.f ? -448.f : b;
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xffffu;
}

// 8 bf16 values as 8 cache elements
__device__ __forceinline__ u32x2 to_fp8(const u32x4& w, float scale) {
  u32x2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t p[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t x = w[2 * i + k];
      p[k] = fp8_pair(bf16_to_f32(x & 0xffffu) / scale, __uint_as_float(x & 0xffff0000u) / scale);
    }
    r[i] = p[0] | (p[1] << 16);
  }
  return r;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) append_kernel(tb_paged_cache c, const uint16_t* __restrict__ k,
                                                          int64_t k_stride, const uint16_t* __restrict__ v,
                                                          int64_t v_stride) {
  typedef typename std::conditional<FP8, uint8_t, uint16_t>::type Elem;
  constexpr int kPiece = 16 / sizeof(Elem);   // positions of one 16-byte store
  constexpr int kRow = D + 16 / sizeof(Elem);  // LDS row of a position: the columns of 16 positions start in other banks
  __shared__ __align__(16) Elem tile[kTile * kRow];

  const int64_t b = blockIdx.z;
  const int head = blockIdx.y;
  const PagedSeq s = paged_seq(c.cu_q, c.kv_len, b, c.total_q, c.table_width * c.page);
  const int n = s.n < c.max_q ? s.n : (int)c.max_q;
  // the new positions that exist, and this workgroup's 64 of them
  const int begin = s.first_pos > 0 ? s.first_pos : 0;
  const int64_t top = (int64_t)s.first_pos + n;
  const int end = top < s.keys ? (int)(top < 0 ? 0 : top) : s.keys;
  const int64_t tile0 = (int64_t)(begin / kTile + (int64_t)blockIdx.x) * kTile;
  if (tile0 >= end) return;
  const int lo = begin > tile0 ? begin - (int)tile0 : 0;
  const int hi = end - tile0 < kTile ? (int)(end - tile0) : kTile;
  const int32_t* row = c.block_table + b * c.table_stride;
  const int shift = __builtin_ctz(c.page);
  const float ks = FP8 && c.k_scale ? c.k_scale[head] : 1.f, vs = FP8 && c.v_scale ? c.v_scale[head] : 1.f;

  for (int i = threadIdx.x; i < kTile * (D / 8); i += kThreads) {
    const int x = i / (D / 8), d = i % (D / 8) * 8;
    if (x < lo || x >= hi) continue;
    const int64_t pos = tile0 + x, token = s.row0 + (pos - s.first_pos);
    const u32x4 kw = *reinterpret_cast<const u32x4*>(k + token * k_stride + head * D + d);
    const u32x4 vw = *reinterpret_cast<const u32x4*>(v + token * v_stride + head * D + d);
    const int page = paged_page(row, c.table_width, c.n_pages, pos >> shift);
    Elem* kd = static_cast<Elem*>(const_cast<void*>(c.k_cache)) +
               (((int64_t)page * c.heads_kv + head) * c.page + (pos & (c.page - 1))) * D + d;
    if constexpr (FP8) {
      if (page >= 0) *reinterpret_cast<u32x2*>(kd) = to_fp8(kw, ks);
      *reinterpret_cast<u32x2*>(tile + x * kRow + d) = to_fp8(vw, vs);
    } else {
      if (page >= 0) *reinterpret_cast<u32x4*>(kd) = kw;
      *reinterpret_cast<u32x4*>(tile + x * kRow + d) = vw;
    }
  }
  __syncthreads();
  constexpr int kPieces = kTile / kPiece;
  for (int i = threadIdx.x; i < D * kPieces; i += kThreads) {
    const int d = i / kPieces, x0 = i % kPieces * kPiece;
    if (x0 + kPiece <= lo || x0 >= hi) continue;
    const int64_t pos = tile0 + x0;  // pages are multiples of 16 positions: a piece lies in one
    const int page = paged_page(row, c.table_width, c.n_pages, pos >> shift);
    if (page < 0) continue;
    Elem* vd = static_cast<Elem*>(const_cast<void*>(c.v_cache)) +
               (((int64_t)page * c.heads_kv + head) * D + d) * c.page + (pos & (c.page - 1));
    if (x0 >= lo && x0 + kPiece <= hi) {
      Elem w[kPiece] __attribute__((aligned(16)));
#pragma unroll
      for (int e = 0; e < kPiece; ++e) w[e] = tile[(x0 + e) * kRow + d];
      *reinterpret_cast<u32x4*>(vd) = *reinterpret_cast<const u32x4*>(w);
    } else {
      for (int e = 0; e < kPiece; ++e)
        if (x0 + e >= lo && x0 + e < hi) vd[e] = tile[(x0 + e) * kRow + d];
    }
  }
}

template <int D>
hipError_t launch(const tb_paged_cache& c, const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                  hipStream_t stream) {
  // a chunk that does not start on a tile reaches into one more
  const dim3 grid((unsigned)((c.max_q + kTile - 1) / kTile + 1), (unsigned)c.heads_kv, (unsigned)c.B);
  if (c.cache_dtype == TB_FP8)
    hipLaunchKernelGGL((append_kernel<D, true>), grid, dim3(kThreads), 0, stream, c, k, k_stride, v, v_stride);
  else
    hipLaunchKernelGGL((append_kernel<D, false>), grid, dim3(kThreads), 0, stream, c, k, k_stride, v, v_stride);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_paged_append(const tb_paged_cache& c, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                               int64_t v_stride, hipStream_t stream) {
  if (c.head_dim == 64) return launch<64>(c, k, k_stride, v, v_stride, stream);
  return launch<128>(c, k, k_stride, v, v_stride, stream);
}

}  // namespace tb
