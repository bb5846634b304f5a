// Host-side argument checks shared by the C ABI sources.  None of them makes
// a HIP call.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tb.h"

namespace tb {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool dtype_ok(int d) { return d == TB_F32 || d == TB_BF16; }
inline size_t dtype_bytes(int d) { return d == TB_F32 ? 4 : 2; }
// bytes of the act8 operand of `elems` activations (4 per element + 1/8 of scales)
inline size_t act8_bytes(size_t elems) { return elems * 4 + elems / 8; }

// [a, a + na) and [b, b + nb) intersect (byte ranges; a null array is empty)
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && pa < pb + nb && pb < pa + na;
}

inline tb_status launched(hipError_t e) { return e == hipSuccess ? TB_OK : TB_ERR_LAUNCH; }

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace tb
