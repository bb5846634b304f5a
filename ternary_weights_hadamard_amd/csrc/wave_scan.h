// Sums of 64-bit values over the lanes of a wave, by DPP moves (an exchange
// through LDS for each step takes several times as long).
#pragma once

#include "tb_common.h"

namespace tb {

// v of the lanes that the DPP control names, 0 where it names none
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T moved(T v) {
  static_assert(sizeof(T) == 8, "two registers");
  const uint64_t w = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)w, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(w >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
}

// inclusive prefix over the lanes of a wave: within rows of 16, then over them
template <typename T>
__device__ __forceinline__ T wave_prefix(T v) {
  v += moved<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
  v += moved<0x112, 0xf>(v);
  v += moved<0x114, 0xf>(v);
  v += moved<0x118, 0xf>(v);
  v += moved<0x142, 0xa>(v);  // lane 15 of rows 0 and 2 to the next row
  v += moved<0x143, 0xc>(v);  // lane 31 to rows 2 and 3
  return v;
}

// a lane's value (the lane is the same for the whole wave) in scalar registers
template <typename T>
__device__ __forceinline__ T of_lane(T v, int lane) {
  static_assert(sizeof(T) == 8, "two registers");
  const uint64_t w = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)w, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(w >> 32), lane);
  return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
}

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
  return of_lane(wave_prefix(v), 63);
}

}  // namespace tb
