// 128-point Walsh-Hadamard butterflies on one block held by 16 consecutive
// lanes, 8 contiguous elements per lane (element 8 * sub + e in v[e] of lane
// `sub`).  xxqk.cn/news/652513 §2 computes the transform as log2(n) rounds of
// (a + b, a - b) butterflies: here the three rounds over element bits 0-2 run
// inside a lane and the four over element bits 3-6 pair lanes (lane ^ 1, 2, 4,
// 8) through DPP and ds_swizzle, so nothing goes through LDS.  The result is
// unnormalised (H v, not H v / sqrt(128)).  All 16 lanes of a block must run
// it together.
#pragma once

#include "tb_common.h"

namespace tb {

constexpr float kInvSqrt128 = 0.08838834764831845f;

// Lane pairs (sub, sub ^ MASK): the lower lane keeps v + p, the upper p - v.
// Both are p + (+-v): the sign flip is one XOR with a per-lane mask, the sum
// one add that can take p straight from the cross-lane read.
template <int MASK>
__device__ __forceinline__ void fwht_lane_round(float (&v)[8], int sub) {
  const uint32_t flip = (sub & MASK) != 0 ? 0x80000000u : 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float p = xor_lane<MASK>(v[e]);
    v[e] = p + __uint_as_float(__float_as_uint(v[e]) ^ flip);
  }
}

__device__ __forceinline__ void fwht128_lanes(float (&v)[8], int sub) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if ((e & h) == 0) {
        const float a = v[e], c = v[e + h];
        v[e] = a + c;
        v[e + h] = a - c;
      }
    }
  }
  fwht_lane_round<1>(v, sub);
  fwht_lane_round<2>(v, sub);
  fwht_lane_round<4>(v, sub);
  fwht_lane_round<8>(v, sub);
}

__device__ __forceinline__ float fused(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
__device__ __forceinline__ double fused(double a, double b, double c) { return __builtin_fma(a, b, c); }

// H v / sqrt(128), in fp32 or in 64 bits.  Between lanes each takes v + p or v -
// p in one operation, which gives the upper lane of a pair its result's negative;
// the lanes of a later pair have the same earlier bits, so the same sign so far,
// and all signs go into the last multiplication.  (In fwht128_lanes a sum stays
// one rounding of the plain butterflies, which other kernels' codes are pinned to.)
template <typename F>
__device__ __forceinline__ void fwht128_normal(F (&v)[8], int sub) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if ((e & h) == 0) {
        const F a = v[e], c = v[e + h];
        v[e] = a + c;
        v[e + h] = a - c;
      }
    }
  }
  const F s1 = sub & 1 ? (F)-1 : (F)1, s2 = sub & 2 ? (F)-1 : (F)1, s4 = sub & 4 ? (F)-1 : (F)1, s8 = sub & 8 ? (F)-1 : (F)1;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = fused(xor_lane<1>(v[e]), s1, v[e]);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = fused(xor_lane<2>(v[e]), s2, v[e]);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = fused(xor_lane<4>(v[e]), s4, v[e]);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = fused(xor_lane<8>(v[e]), s8, v[e]);
  const F f = (s1 * s2) * (s4 * s8) * (F)0x1.6a09e667f3bcdp-4;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= f;
}

}  // namespace tb
