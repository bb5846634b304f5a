// The boundary between two blocks of a decoder layer in one launch: the norm
// after a block, its gate, residual scale and residual, and the norm before
// the next block, with the rotations of the products on both sides
// (include/tb.h, tb_block_norm).
//
// A row lives in one workgroup's registers, 8 contiguous channels per lane and
// pass, so that 16 consecutive lanes hold a 128-block and the rotations are
// the in-register butterflies of fwht_lanes.h.  Each norm is one sum over the
// row: a wave reduction, then one LDS exchange between the waves.
#include "act8.h"
#include "fwht_lanes.h"
#include "tb_common.h"
#include "tb_launch.h"

namespace tb {

namespace {

__device__ __forceinline__ void load8(const void* p, int dtype, int64_t i, float (&v)[8]) {
  if (dtype == TB_BF16) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = bf16_to_f32(w[e] & 0xffffu);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  } else {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
    const f32x4 a = q[0], c = q[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = c[e];
    }
  }
}

__device__ __forceinline__ void store8(void* p, int dtype, int64_t i, const float (&v)[8]) {
  if (dtype == TB_BF16) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = f32_to_bf16_rne(v[2 * e]) | (f32_to_bf16_rne(v[2 * e + 1]) << 16);
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
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < waves; ++w) s += part[w];
  return s;
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
  }
}

// NP passes of 8 channels per lane cover the row.  Lanes past its end hold
// zeros and take part in the reductions and butterflies only (whole 16-lane
// groups of them: C is a multiple of 128).
template <int NP>
__global__ void __launch_bounds__(1024) block_norm_kernel(tb_block_norm_args a) {
  __shared__ float part[2][16];
  const int sub = threadIdx.x & 15;
  const float inv_c = 1.f / (float)a.C;
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const int64_t base = r * a.C;
    int col[NP];
    bool live[NP];
    float h[NP][8], u[NP][8];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      col[n] = (n * (int)blockDim.x + (int)threadIdx.x) * 8;
      live[n] = col[n] < a.C;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[n][e] = u[n][e] = 0.f;
      if (live[n] && a.resid) load8(a.resid, a.h_dtype, base + col[n], h[n]);
    }
    if (a.y) {
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        if (!live[n]) continue;
        load8(a.y, a.y_dtype, base + col[n], u[n]);
        for (int p = 1; p < a.parts; ++p) {
          float t[8];
          load8(a.y, a.y_dtype, ((int64_t)p * a.rows) * a.C + base + col[n], t);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[n][e] += t[e];
        }
      }
      if (a.rotate_in) rotate(u, sub);
      float inv = a.alpha;
      if (a.w_post) {
        inv *= rsqrtf(workgroup_sum(sum_squares(u), part[turn]) * inv_c + a.eps);
        turn ^= 1;
      }
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        if (!live[n]) continue;
        float w[8], g[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = g[e] = 1.f;
        if (a.w_post) load8(a.w_post, a.w_dtype, col[n], w);
        if (a.gate) load8(a.gate, a.gate_dtype, r / a.rows_per_gate * a.C + col[n], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[n][e] = fmaf(u[n][e] * inv, w[e] * g[e], h[n][e]);
      }
    }
    if (a.h) {
#pragma unroll
      for (int n = 0; n < NP; ++n)
        if (live[n]) store8(a.h, a.h_dtype, base + col[n], h[n]);
    }
    if (!a.z) continue;
    const float inv = rsqrtf(workgroup_sum(sum_squares(h), part[turn]) * inv_c + a.eps);
    turn ^= 1;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 0.f;
      if (live[n]) load8(a.w_pre, a.w_dtype, col[n], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[n][e] = h[n][e] * inv * w[e];
    }
    if (a.rotate_out) rotate(h, sub);
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      if (a.z_dtype == TB_ACT8) {
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
    }
  }
}

template <int NP>
hipError_t launch(const tb_block_norm_args& a, hipStream_t stream) {
  const int64_t lanes = (a.C / 8 + NP - 1) / NP;
  const unsigned threads = (unsigned)((lanes + 63) / 64 * 64);
  const int64_t cap = 1 << 20;
  hipLaunchKernelGGL((block_norm_kernel<NP>), dim3((unsigned)(a.rows < cap ? a.rows : cap)), dim3(threads), 0, stream,
                     a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const tb_block_norm_args& a, hipStream_t stream) {
  if (a.C <= 8 * 1024) return launch<1>(a, stream);
  if (a.C <= 2 * 8 * 1024) return launch<2>(a, stream);
  return launch<4>(a, stream);
}

}  // namespace tb
