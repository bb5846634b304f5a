// New keys and values into the paged cache (include/tb.h, tb_paged_append).
//
// K pages are [position][d], so a token's row is copied as it is.  V pages are
// [d][position] (the attention loads 8 or 16 positions of one d as a matrix
// operand), so values are turned: a workgroup takes 64 positions of one head; a
// thread loads 8 channels of the positions that fill one word, so that the
// conversion to the cache's type puts them side by side, and from LDS each d's
// run of positions is written in 16-byte pieces where all of a piece is new.
//
// Bound by the chain lengths - entry - load - convert - store, of which a chunk
// has one round (4 x 128..2048 tokens of 8 heads to e4m3, 24.5 MB: 12.9 us, 1.9
// TB/s) and a step little else (16 tokens of 8 heads: 5.8 us).
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

// x / scale, correctly rounded, for a scale whose reciprocal and products stay
// far from the ends of fp32: the rounded quotient by the reciprocal, corrected
// by its remainder once (exact but for quotients that e4m3 rounds to 0).  3 operations in place of about 10 of
// the general division.  Quotients past
// 512 are cut there before the correction, so that none of it overflows; NaN
// and infinities come through by the remainder.
struct Quotient {
  float scale, inverse;
  bool plain;
  __device__ explicit Quotient(float s) : scale(s), inverse(1.f / s) { plain = s >= 0x1p-60f && s <= 0x1p60f; }
  __device__ float operator()(float x) const {
    if (!plain) return x / scale;
    const float q = __builtin_amdgcn_fmed3f(x * inverse, -512.f, 512.f);
    return __builtin_fmaf(-__builtin_fmaf(q, scale, -x), inverse, q);  // signs so that -0 stays -0
  }
};

// channels 2w and 2w + 1 of a row of bf16
__device__ __forceinline__ float channel(const u32x4& w, int d) {
  return d & 1 ? __uint_as_float(w[d >> 1] & 0xffff0000u) : bf16_to_f32(w[d >> 1] & 0xffffu);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) append_kernel(tb_paged_cache c, const uint16_t* __restrict__ k,
                                                          int64_t k_stride, const uint16_t* __restrict__ v,
                                                          int64_t v_stride) {
  typedef typename std::conditional<FP8, uint8_t, uint16_t>::type Elem;
  constexpr int kPiece = 16 / sizeof(Elem);   // positions of one 16-byte store
  constexpr int kPieces = kTile / kPiece;     // of a d's 64 positions
  constexpr int kWord = 4 / sizeof(Elem);     // positions of one word
  constexpr int kRow = kTile / kWord + 4;     // words in LDS for a d
  // Threads write one word at 8 d's each; a piece's place is moved by the d, so
  // that those of a wave spread over the banks.
  __shared__ __align__(16) uint32_t tile[D * kRow];
  auto place = [](int d, int piece) { return d * kRow + 4 * (piece ^ ((d >> 4) & (kPieces - 1))); };

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
  const Quotient ks(FP8 && c.k_scale ? c.k_scale[head] : 1.f), vs(FP8 && c.v_scale ? c.v_scale[head] : 1.f);

#pragma unroll
  for (int i = threadIdx.x; i < kTile / kWord * (D / 8); i += kThreads) {
    const int x0 = i / (D / 8) * kWord, d = i % (D / 8) * 8;
    if (x0 + kWord <= lo || x0 >= hi) continue;
    const int64_t pos = tile0 + x0;
    u32x4 kw[kWord], vw[kWord];
#pragma unroll
    for (int e = 0; e < kWord; ++e) {
      kw[e] = vw[e] = u32x4{0u, 0u, 0u, 0u};
      if (x0 + e < lo || x0 + e >= hi) continue;
      const int64_t token = s.row0 + (pos + e - s.first_pos);
      kw[e] = *reinterpret_cast<const u32x4*>(k + token * k_stride + head * D + d);
      vw[e] = *reinterpret_cast<const u32x4*>(v + token * v_stride + head * D + d);
    }
    // pages are multiples of 16 positions: these lie in one
    const int page = paged_page(row, c.table_width, c.n_pages, pos >> shift);
    if (page < 0) continue;
    Elem* kd = static_cast<Elem*>(const_cast<void*>(c.k_cache)) +
               (((int64_t)page * c.heads_kv + head) * c.page + (pos & (c.page - 1))) * D + d;
#pragma unroll
    for (int e = 0; e < kWord; ++e) {
      if (x0 + e < lo || x0 + e >= hi) continue;
      if constexpr (FP8) {
        u32x2 w;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[h] = fp8_pair(ks(channel(kw[e], 4 * h)), ks(channel(kw[e], 4 * h + 1))) |
                 fp8_pair(ks(channel(kw[e], 4 * h + 2)), ks(channel(kw[e], 4 * h + 3))) << 16;
        *reinterpret_cast<u32x2*>(kd + e * D) = w;
      } else {
        *reinterpret_cast<u32x4*>(kd + e * D) = kw[e];
      }
    }
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      uint32_t w;
      if constexpr (FP8)
        w = fp8_pair(vs(channel(vw[0], y)), vs(channel(vw[1], y))) |
            fp8_pair(vs(channel(vw[2], y)), vs(channel(vw[3], y))) << 16;
      else
        w = y & 1 ? (vw[0][y >> 1] >> 16) | (vw[1][y >> 1] & 0xffff0000u)
                  : (vw[0][y >> 1] & 0xffffu) | (vw[1][y >> 1] << 16);
      tile[place(d + y, x0 / kPiece) + x0 % kPiece / kWord] = w;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = threadIdx.x; i < D * kPieces; i += kThreads) {
    const int d = i / kPieces, piece = i % kPieces, x0 = piece * kPiece;
    if (x0 + kPiece <= lo || x0 >= hi) continue;
    const int64_t pos = tile0 + x0;  // a piece lies in one page too
    const int page = paged_page(row, c.table_width, c.n_pages, pos >> shift);
    if (page < 0) continue;
    Elem* vd = static_cast<Elem*>(const_cast<void*>(c.v_cache)) +
               (((int64_t)page * c.heads_kv + head) * D + d) * c.page + (pos & (c.page - 1));
    const uint32_t* from = tile + place(d, piece);
    if (x0 >= lo && x0 + kPiece <= hi) {
      *reinterpret_cast<u32x4*>(vd) = *reinterpret_cast<const u32x4*>(from);
    } else {
      for (int e = 0; e < kPiece; ++e)
        if (x0 + e >= lo && x0 + e < hi) vd[e] = reinterpret_cast<const Elem*>(from)[e];
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
