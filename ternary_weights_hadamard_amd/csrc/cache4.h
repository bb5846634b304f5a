// Values of 4-bit codes (include/tb.h, TB_INT4).  A code in the high half of a
// byte, below the byte 0x54, is the fp16 number 64 + code (64 has its unit in
// bit 4 of the significand): bytes are masked and spread, eight codes by three
// operations and four permutes, and then multiplied with the scale and added to
// the offset two at a time.
#pragma once

#include "tb_common.h"

namespace tb {

struct Nibbles {
  uint32_t low, high;  // the codes of each byte's low and high half, in the high half
};
__device__ __forceinline__ Nibbles nibbles(uint32_t w) { return Nibbles{w << 4 & 0xf0f0f0f0u, w & 0xf0f0f0f0u}; }

// 64 + code, of bytes 0 and 1 (or 2 and 3), times the scales, plus the offsets
template <int PAIR>
__device__ __forceinline__ f16x2 pair4(uint32_t codes, f16x2 scale, f16x2 offset) {
  const uint32_t w = __builtin_amdgcn_perm(0x54545454u, codes, PAIR == 0 ? 0x04010400u : 0x04030402u);
  return __builtin_elementwise_fma(__builtin_bit_cast(f16x2, w), scale, offset);
}

__device__ __forceinline__ f16x8 join4(f16x2 a, f16x2 b, f16x2 c, f16x2 d) {
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Eight channels of one position; `so` its scale and, above it, its offset.
__device__ __forceinline__ f16x8 channels4(uint32_t w, uint32_t so) {
  const f16x2 x = __builtin_bit_cast(f16x2, so), s = {x[0], x[0]}, o = {x[1], x[1]};
  const Nibbles n = nibbles(w);
  return join4(pair4<0>(n.low, s, o), pair4<1>(n.low, s, o), pair4<0>(n.high, s, o), pair4<1>(n.high, s, o));
}

// One channel of eight positions, from two words' low (or high) codes and the
// positions' scales and offsets.
__device__ __forceinline__ f16x8 positions4(uint32_t w0, uint32_t w1, const u32x4& scales, const u32x4& offsets) {
  f16x2 s[4], o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // by values of their own: a bit cast of a vector's element takes its first one
    const uint32_t sw = scales[i], ow = offsets[i];
    s[i] = __builtin_bit_cast(f16x2, sw);
    o[i] = __builtin_bit_cast(f16x2, ow);
  }
  return join4(pair4<0>(w0, s[0], o[0]), pair4<1>(w0, s[1], o[1]), pair4<0>(w1, s[2], o[2]), pair4<1>(w1, s[3], o[3]));
}

}  // namespace tb
