// What writes the paged cache's codes: bf16 pairs taken apart, e4m3 and 4-bit
// roundings.
#pragma once

#include "tb_common.h"

namespace tb {

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

// The scale and offset of a position's channels in 4 bits (include/tb.h,
// TB_INT4), and its codes: a group of LANES = D / 8 consecutive lanes holds a
// position, 8 channels a lane, in 64 bits, or in 32 if they are exact there.
// All of it is found in 32 bits first.  Scale and offset round what has 24 bits
// or more to 11: by 32 alone some rows of 65536 would get another scale, and with
// it other values in every channel.  But rounding and clamping are monotone: where
// both ends of the interval of what 32 bits may have lost give the same fp16, 64
// give it too; where they do not, 64 decide.  A code is found as x / scale + away
// with away = -offset / scale: of a quotient that is at most 80, less than 2^-15 is
// lost, and of away and of x / scale, which far from 0 are large and cancel, 2^-24
// each.  Only one that may be that near to the middle between two codes is
// looked at in 64.
struct Codes4 {
  uint32_t word;   // byte i: channels i (low) and i + 4 of the lane's eight
  uint32_t scale;  // fp16 bits: scale, and offset above it
};
constexpr float kLimit4 = 4096.f;

__device__ __forceinline__ float least(float a, float b) { return __builtin_fminf(a, b); }
__device__ __forceinline__ float most(float a, float b) { return __builtin_fmaxf(a, b); }
__device__ __forceinline__ double least(double a, double b) { return __builtin_fmin(a, b); }
__device__ __forceinline__ double most(double a, double b) { return __builtin_fmax(a, b); }

// The least and the largest channel of the group, first limited.
template <int LANES, typename F>
__device__ __forceinline__ void ends4(const F (&x)[8], F& lo, F& hi) {
  lo = (F)kLimit4;
  hi = -(F)kLimit4;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lo = least(lo, x[e]);
    hi = most(hi, x[e]);
  }
  auto join = [&](F l, F h) {
    lo = least(lo, l);
    hi = most(hi, h);
  };
  join(xor_lane<1>(lo), xor_lane<1>(hi));
  join(xor_lane<2>(lo), xor_lane<2>(hi));
  join(xor_lane<4>(lo), xor_lane<4>(hi));
  if constexpr (LANES == 16) join(xor_lane<8>(lo), xor_lane<8>(hi));
  lo = most(lo, -(F)kLimit4);
  hi = least(hi, (F)kLimit4);
}

template <int LANES, typename F>
__device__ __forceinline__ Codes4 codes4(const F (&x)[8]) {
  bool nan = false;
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    y[e] = (float)x[e];
    nan = nan || y[e] != y[e];
  }
  float lo, hi;
  ends4<LANES>(y, lo, hi);
  // 2^-21 is several times what the operations here lose, 2^-24 of the larger end
  // what x did on its way to 32 bits
  const float narrow = sizeof(F) == 4 ? 0.f : most(fabsf(lo), fabsf(hi)) * 0x1p-24f;
  const float step = (hi - lo) * (1.f / 15.f), step_off = __builtin_fmaf(step, 0x1p-21f, narrow * 0.14f);
  _Float16 sh = (_Float16)(step - step_off);
  const float low = __builtin_fmaf(-64.f, (float)sh, lo), low_off = __builtin_fmaf(fabsf(low), 0x1p-21f, narrow);
  _Float16 oh = (_Float16)(low - low_off);
  const bool sure = !nan && sh > (_Float16)0.f && sh == (_Float16)(step + step_off) && oh == (_Float16)(low + low_off) &&
                    oh != (_Float16)0.f;
  const int lane = threadIdx.x & 63;
  const uint64_t group = ((uint64_t)1 << LANES) - 1;
  if ((__ballot(!sure) >> (lane & ~(LANES - 1)) & group) != 0) {
    if ((__ballot(nan) >> (lane & ~(LANES - 1)) & group) != 0) return Codes4{0u, 0x7e007e00u};
    F l, h;
    ends4<LANES>(x, l, h);
    sh = (_Float16)(((double)h - (double)l) / 15.0);
    oh = (_Float16)((double)l - 64.0 * (double)sh);
  }
  Codes4 r;
  r.word = 0u;
  r.scale = (uint32_t)__builtin_bit_cast(uint16_t, sh) | (uint32_t)__builtin_bit_cast(uint16_t, oh) << 16;
  if (!(sh > (_Float16)0.f)) return r;
  const float inverse = 1.f / (float)sh, away = -(float)oh * inverse;
  float n[8], far = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float q = __builtin_fmaf(most(least(y[e], kLimit4), -kLimit4), inverse, away);
    n[e] = __builtin_rintf(q);
    far = __builtin_fmaxf(far, fabsf(q - n[e]));
  }
  if (far > 0.5f - __builtin_fmaf(fabsf(away), 0x1p-22f, 0x1p-15f)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double limited = most(least((double)x[e], (double)kLimit4), -(double)kLimit4);
      n[e] = (float)__builtin_rint((limited - (double)oh) / (double)sh);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    r.word |= (uint32_t)(int)__builtin_amdgcn_fmed3f(n[e] - 64.f, 0.f, 15.f) << (8 * (e & 3) + (e & 4));
  return r;
}

}  // namespace tb
