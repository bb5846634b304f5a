// The boundary between two blocks of a decoder layer in one launch: the norm
// after a block, its gate, residual scale and residual, and the norm before
// the next block, with the rotations of the products on both sides
// (include/tb.h, tb_block_norm).
//
// A row lives in one workgroup's registers, 8 contiguous channels per lane and
// pass, so that 16 consecutive lanes hold a 128-block and the rotations are
// the in-register butterflies of fwht_lanes.h.  Each norm is one sum over the
// row: a wave reduction in registers, then one LDS exchange between the waves.
//
// What bounds it: HBM for many rows (2048 rows of 5120, y, gate and residual
// read, h and z written in bf16, 105 MB: 22.9 us, 4.6 TB/s), the chain load -
// sum - sum - store for a few (one row: 4.8 us).  So the arrays of rows are
// loaded before the first sum, raw, and widened when used, and the weights of a
// norm before its sum is known.
#include "act8.h"
#include "fwht_lanes.h"
#include "tb_common.h"
#include "tb_launch.h"

namespace tb {

namespace {

// 8 channels as they are stored: four words of bf16 or eight of fp32.
template <int DTYPE>
struct Raw {
  u32x4 a[DTYPE == TB_BF16 ? 1 : 2];
};

template <int DTYPE>
__device__ __forceinline__ Raw<DTYPE> load_raw(const void* p, int64_t i) {
  Raw<DTYPE> r;
  const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const char*>(p) + i * (DTYPE == TB_BF16 ? 2 : 4));
  r.a[0] = q[0];
  if constexpr (DTYPE == TB_F32) r.a[1] = q[1];
  return r;
}

template <int DTYPE>
__device__ __forceinline__ void widen(const Raw<DTYPE>& r, float (&v)[8]) {
  if constexpr (DTYPE == TB_BF16) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = bf16_to_f32(r.a[0][e] & 0xffffu);
      v[2 * e + 1] = __uint_as_float(r.a[0][e] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r.a[e >> 2][e & 3]);
  }
}

// The same with the dtype known at run time (uniform): weights and gates.
struct RawAny {
  u32x4 a, b;
};

__device__ __forceinline__ RawAny load_any(const void* p, int dtype, int64_t i) {
  RawAny r;
  if (dtype == TB_BF16) {
    r.a = load_raw<TB_BF16>(p, i).a[0];
    r.b = u32x4{0u, 0u, 0u, 0u};
  } else {
    const Raw<TB_F32> f = load_raw<TB_F32>(p, i);
    r.a = f.a[0];
    r.b = f.a[1];
  }
  return r;
}

__device__ __forceinline__ void widen(const RawAny& r, int dtype, float (&v)[8]) {
  if (dtype == TB_BF16) widen(Raw<TB_BF16>{{r.a}}, v);
  else widen(Raw<TB_F32>{{r.a, r.b}}, v);
}

// two values as bf16, to nearest even (v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  bf16x2 r;
  r[0] = (__bf16)lo;
  r[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ void store8(void* p, int dtype, int64_t i, const float (&v)[8]) {
  if (dtype == TB_BF16) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = w;
  } else {
    f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + i);
    q[0] = f32x4{v[0], v[1], v[2], v[3]};
    q[1] = f32x4{v[4], v[5], v[6], v[7]};
  }
}

// Sum of `v` over the workgroup, the same in every lane.  `part` holds one
// float per wave; consecutive calls must alternate between two arrays (a wave
// may enter the next call while another still reads this one's parts).
__device__ __forceinline__ float workgroup_sum(float v, float* part) {
  v += xor_lane<1>(v);
  v += xor_lane<2>(v);
  v += xor_lane<4>(v);
  v += xor_lane<8>(v);
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  float lower, upper;
  swap_halves(v, lower, upper);
  v = lower + upper;
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  // lane w of each 16 holds wave w's part
  const int w = threadIdx.x & 15;
  v = w < waves ? part[w] : 0.f;
  v += xor_lane<1>(v);
  v += xor_lane<2>(v);
  v += xor_lane<4>(v);
  return v + xor_lane<8>(v);
}

// Passes one after another: interleaved, they would need the registers of all.
template <int NP>
__device__ __forceinline__ void pass_end() {
  if constexpr (NP > 1) __builtin_amdgcn_sched_barrier(0);
}

template <int NP>
__device__ __forceinline__ float sum_squares(const float (&v)[NP][8]) {
  float s = 0.f;
#pragma unroll
  for (int n = 0; n < NP; ++n)
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(v[n][e], v[n][e], s);
  return s;
}

template <int NP>
__device__ __forceinline__ void rotate(float (&v)[NP][8], int sub) {
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    fwht128_lanes(v[n], sub);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[n][e] *= kInvSqrt128;
    pass_end<NP>();
  }
}

// NP passes of 8 channels per lane cover the row.  Lanes past its end hold
// zeros and take part in the reductions and butterflies only (whole 16-lane
// groups of them: C is a multiple of 128).
// T: most threads of a workgroup.  Long rows are loaded as they are used.  No
// loop over rows: in one, the compiler keeps the weights of all passes in
// registers from row to row and spills the rows (2048 rows of 5120: 42 us at
// 80 registers with spills, 30 us at 94 without, in a loop).
template <int NP, int T, int YD, int HD, bool ACT8>
__global__ void __launch_bounds__(T) block_norm_kernel(tb_block_norm_args a) {
  constexpr bool kEarly = NP <= 2;
  __shared__ float part[2][16];
  const int sub = threadIdx.x & 15;
  const float inv_c = 1.f / (float)a.C;
  const int C = (int)a.C;
  int turn = 0;
  int col[NP];
  bool live[NP];
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    col[n] = (n * (int)blockDim.x + (int)threadIdx.x) * 8;
    live[n] = col[n] < C;
  }
  const int64_t r = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (r >= a.rows) return;
  const int64_t base = r * C;
  // one gate for all rows, or one for each, need no division
  const int64_t gate_row = a.rows_per_gate == 1 ? r : a.rows_per_gate >= a.rows ? 0 : r / a.rows_per_gate;
  Raw<YD> yr[NP];
  Raw<HD> hr[NP];
  RawAny gr[NP], w[NP];
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    if (!live[n]) continue;
    if (!kEarly) continue;
    if (a.y) yr[n] = load_raw<YD>(a.y, base + col[n]);
    if (a.resid) hr[n] = load_raw<HD>(a.resid, base + col[n]);
    if (a.gate) gr[n] = load_any(a.gate, a.gate_dtype, gate_row * C + col[n]);
  }
  float h[NP][8];
  if (a.y) {
    float u[NP][8];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[n][e] = 0.f;
      if (!live[n]) continue;
      if (kEarly && a.w_post) w[n] = load_any(a.w_post, a.w_dtype, col[n]);
      if (!kEarly) yr[n] = load_raw<YD>(a.y, base + col[n]);
      widen(yr[n], u[n]);
      if constexpr (YD == TB_F32) {
        // parts in order, the loads of four before their sum
        for (int k = 1; k < a.parts; k += 4) {
          Raw<TB_F32> p[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (k + x < a.parts) p[x] = load_raw<TB_F32>(a.y, (int64_t)(k + x) * a.rows * C + base + col[n]);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (k + x < a.parts) {
              float t[8];
              widen(p[x], t);
#pragma unroll
              for (int e = 0; e < 8; ++e) u[n][e] += t[e];
            }
        }
      }
      pass_end<NP>();
    }
    if (a.rotate_in) rotate(u, sub);
    float inv = a.alpha;
    if (a.w_post) {
      inv *= rsqrtf(workgroup_sum(sum_squares(u), part[turn]) * inv_c + a.eps);
      turn ^= 1;
    }
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      float f[8], g[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = g[e] = 1.f, h[n][e] = 0.f;
      if (!live[n]) continue;
      if (!kEarly) {
        if (a.resid) hr[n] = load_raw<HD>(a.resid, base + col[n]);
        if (a.gate) gr[n] = load_any(a.gate, a.gate_dtype, gate_row * C + col[n]);
        if (a.w_post) w[n] = load_any(a.w_post, a.w_dtype, col[n]);
      }
      if (a.resid) widen(hr[n], h[n]);
      if (a.w_post) widen(w[n], a.w_dtype, f);
      if (a.gate) widen(gr[n], a.gate_dtype, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[n][e] = fmaf(u[n][e] * inv, f[e] * g[e], h[n][e]);
      pass_end<NP>();
    }
  } else {
#pragma unroll
    for (int n = 0; n < NP; ++n) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[n][e] = 0.f;
      if (!kEarly && live[n]) hr[n] = load_raw<HD>(a.resid, base + col[n]);
      if (live[n]) widen(hr[n], h[n]);
    }
  }
  if (kEarly && a.z) {
#pragma unroll
    for (int n = 0; n < NP; ++n)
      if (live[n]) w[n] = load_any(a.w_pre, a.w_dtype, col[n]);
  }
  if (a.h) {
#pragma unroll
    for (int n = 0; n < NP; ++n)
      if (live[n]) {
        store8(a.h, HD, base + col[n], h[n]);
        pass_end<NP>();
      }
  }
  if (!a.z) return;
  const float inv = rsqrtf(workgroup_sum(sum_squares(h), part[turn]) * inv_c + a.eps);
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
    if (!kEarly && live[n]) w[n] = load_any(a.w_pre, a.w_dtype, col[n]);
    if (live[n]) widen(w[n], a.w_dtype, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[n][e] = h[n][e] * inv * f[e];
    pass_end<NP>();
  }
  if (a.rotate_out) rotate(h, sub);
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    if constexpr (ACT8) {
      // the operand's value and scale bytes of block `blk` of all rows' blocks
      uint32_t bits[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) bits[e] = f32_to_bf16_rne(h[n][e]);
      uint8_t* act = static_cast<uint8_t*>(a.z);
      const int64_t blk = live[n] ? (base + col[n]) / kBlock : 0;
      act8_encode_store(bits, sub, act + blk * 512, act + a.rows * a.C * 4 + blk * 16, live[n]);
    } else if (live[n]) {
      store8(a.z, a.z_dtype, base + col[n], h[n]);
    }
    pass_end<NP>();
  }
}

template <int NP, int T>
hipError_t launch(const tb_block_norm_args& a, hipStream_t stream) {
  const int64_t lanes = (a.C / 8 + NP - 1) / NP;
  // a workgroup per row; the row of workgroup (x, y) is y * gridDim.x + x
  const int64_t cap = 1 << 20;
  const dim3 grid((unsigned)(a.rows < cap ? a.rows : cap), (unsigned)((a.rows + cap - 1) / cap));
  const dim3 block((unsigned)((lanes + 63) / 64 * 64));
  const bool yb = a.y_dtype == TB_BF16, hb = a.h_dtype == TB_BF16;
#define TB_NORM(Y, H)                                                                                   \
  do {                                                                                                  \
    if (a.z_dtype == TB_ACT8) hipLaunchKernelGGL((block_norm_kernel<NP, T, Y, H, true>), grid, block, 0, stream, a); \
    else hipLaunchKernelGGL((block_norm_kernel<NP, T, Y, H, false>), grid, block, 0, stream, a);           \
  } while (0)
  if (yb && hb) TB_NORM(TB_BF16, TB_BF16);
  else if (yb) TB_NORM(TB_BF16, TB_F32);
  else if (hb) TB_NORM(TB_F32, TB_BF16);
  else TB_NORM(TB_F32, TB_F32);
#undef TB_NORM
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const tb_block_norm_args& a, hipStream_t stream) {
  // As many lanes as a row has work for, up to 640: with two passes by half the
  // lanes 2048 rows of 5120 take 26.8 us and one row 6.0 us.
  if (a.C <= 8 * 640) return launch<1, 640>(a, stream);
  if (a.C <= 2 * 8 * 512) return launch<2, 512>(a, stream);
  if (a.C <= 4 * 8 * 512) return launch<4, 512>(a, stream);
  return launch<8, 512>(a, stream);
}

}  // namespace tb
