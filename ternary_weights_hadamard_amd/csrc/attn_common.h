// What the attention kernels share: operand conversions, the softmax
// statistics' helpers, and the product with values that may not be finite.
#pragma once

#include "paged.h"
#include "tb_common.h"

namespace tb {

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// What the weights of a row with maximum m (log2 units) are relative to.  As
// fp16 (e4m3 caches) weights up to 1 would lose bits below 2^-14 and be 0 below
// 2^-25, while the row's sum still counts them: beside one score 14 (in units
// of e) above the others, whose value is small, nothing of these would be left.
// Relative to `ROOM` less than the maximum they use all of fp16's range.  Where
// fp32 cannot tell m from m - ROOM they stay relative to m.
template <int ROOM>
__device__ __forceinline__ float weight_reference(float m) {
  return ROOM > 0 && fabsf(m) < 0x1p20f ? m - (float)ROOM : m;
}

// 8 e4m3 bytes widened to bf16 / fp16: both hold every e4m3 value exactly
__device__ __forceinline__ bf16x8 fp8_to_bf16(const u32x2& w) {
  bf16x8 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, true);
    r[4 * i] = a[0];
    r[4 * i + 1] = a[1];
    r[4 * i + 2] = b[0];
    r[4 * i + 3] = b[1];
  }
  return r;
}

__device__ __forceinline__ f16x8 fp8_to_f16(const u32x2& w) {
  f16x8 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i], 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i], 1.0f, true);
    r[4 * i] = a[0];
    r[4 * i + 1] = a[1];
    r[4 * i + 2] = b[0];
    r[4 * i + 3] = b[1];
  }
  return r;
}

// Values that are not finite must reach only the tokens that see their
// position, and a matrix instruction multiplies every value with every token's
// weight, 0 where the token does not see it.  In the rare tile where both
// occur, two products with 1 in the places of +inf (or NaN) and -inf (or NaN)
// first count what each token sees of them, and the values then go in with
// these elements replaced by 0.  An infinity that all tokens see is one in each
// sum, but its product is NaN with a weight that has rounded to 0 (or with the
// low part of one).  Such sums are found when a part of the work is done; it is
// then done again with the values of all tiles taken out and counted, and
// keep_infinity joins the parts.  (e4m3 has no infinities, and NaN stays NaN.)
template <typename V8>
struct Nonfinite {
  V8 up, down;
};

template <typename V8>
__device__ __forceinline__ Nonfinite<V8> take_nonfinite(V8& v) {
  Nonfinite<V8> r;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float f = (float)v[e];
    const bool fin = fabsf(f) < __builtin_inff();
    r.up[e] = !fin && !(f < 0.f) ? 1.f : 0.f;
    r.down[e] = !fin && !(f > 0.f) ? 1.f : 0.f;
    if (!fin) v[e] = 0.f;
  }
  return r;
}

// what the counts of seen infinities and NaN add to a sum: +inf - inf is NaN
__device__ __forceinline__ float nonfinite_sum(float up, float down) {
  return (up > 0.f ? __builtin_inff() : 0.f) + (down > 0.f ? -__builtin_inff() : 0.f);
}

// A factor of a sum that may hold an infinity: never 0.
__device__ __forceinline__ float keep_infinity(float f) { return fmaxf(f, 1.17549435e-38f); }

template <typename V>
__device__ __forceinline__ bool any_nonfinite(const V& v, int n) {
  bool bad = false;
#pragma unroll
  for (int e = 0; e < n; ++e) bad = bad || !(fabsf(v[e]) < __builtin_inff());
  return bad;
}

// any element of 8 bf16 (four words) infinite or NaN
__device__ __forceinline__ bool any_nonfinite_bf16(const u32x4& w) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    bad = bad || (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
  return bad;
}

// any element of 8 fp16 (four words) infinite or NaN
__device__ __forceinline__ bool any_nonfinite_f16(const u32x4& w) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    bad = bad || (w[i] & 0x7c00u) == 0x7c00u || (w[i] & 0x7c000000u) == 0x7c000000u;
  return bad;
}

// any of 16 e4m3 bytes NaN (0x7f or 0xff; e4m3 has no infinity)
__device__ __forceinline__ bool any_nonfinite_fp8(const u32x4& w) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) bad = bad || ((w[i] >> (8 * e)) & 0x7fu) == 0x7fu;
  return bad;
}

// 16 e4m3 bytes with NaN replaced by 0
__device__ __forceinline__ u32x4 drop_nonfinite_fp8(u32x4 w) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (((w[i] >> (8 * e)) & 0x7fu) == 0x7fu) w[i] &= ~(0xffu << (8 * e));
  return w;
}

}  // namespace tb
