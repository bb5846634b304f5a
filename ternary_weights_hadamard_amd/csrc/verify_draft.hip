// Verification of drafted tokens against the target's probabilities, from
// given random numbers (include/tb.h, tb_verify_draft).
//
// What has to be read is one row of p and one of q per sequence: the row where
// the first token is not kept.  A first launch decides that row (each
// workgroup for itself: a gather of at most TB_MAX_DRAFT pairs) and sums its
// slice of the weights; a second one, a workgroup per sequence, adds the
// slices' sums in order, finds the slice that holds u_next * sum and then the
// token in it.  Differences and sums are in 64 bits, so that which token an
// edge falls to does not depend on how the sum is split.
#include "tb_common.h"
#include "tb_launch.h"

namespace tb {

namespace {

constexpr int kThreads = 256;

// the weights' sums of one slice: of max(p - q, 0), and of p alone
struct SliceSum {
  double rest, target;
};

__device__ __forceinline__ float load1(const void* p, int dtype, int64_t i) {
  if (dtype == TB_BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

// a weight that is not positive and finite counts as 0
__device__ __forceinline__ double weight(double w) { return w > 0.0 && w < __builtin_huge_val() ? w : 0.0; }

struct Row {
  int64_t p, q;     // first elements of the row in p and in q
  int64_t seq_at;   // first draft of the sequence
  int T, kept;      // drafts looked at, and how many of them are kept
  int drop;         // certain drafter: the token that is not kept (else -1)
  bool rest;        // weights max(p - q, 0), not p
};

// Every lane of the wave calls this with the same b; the same answer in each.
__device__ __forceinline__ Row find_row(const tb_verify_draft_args& a, int64_t b) {
  Row r;
  const int64_t lo = min(max((int64_t)a.cu_draft[b], (int64_t)0), a.total);
  const int64_t hi = min(max((int64_t)a.cu_draft[b + 1], lo), a.total);
  r.seq_at = lo;
  r.T = (int)min(hi - lo, (int64_t)a.max_draft);
  const int j = threadIdx.x & 63;
  bool keep = false;
  if (j < r.T) {
    const int d = a.drafts[lo + j];
    if (d >= 0 && d < a.vocab) {
      const double pd = load1(a.p, a.p_dtype, (lo + b + j) * a.p_stride + d);
      const double qd = a.q ? (double)load1(a.q, a.q_dtype, (lo + j) * a.q_stride + d) : 1.0;
      keep = (double)a.u[lo + j] * qd < pd;
    }
  }
  const uint64_t lost = ~__ballot(keep);
  r.kept = lost == 0 ? 64 : __builtin_ctzll(lost);
  r.rest = r.kept < r.T;
  r.p = (lo + b + r.kept) * a.p_stride;
  r.q = r.rest ? (lo + r.kept) * a.q_stride : 0;
  r.drop = r.rest && !a.q ? a.drafts[lo + r.kept] : -1;
  return r;
}

__device__ __forceinline__ void weights_at(const tb_verify_draft_args& a, const Row& r, int64_t v, double& rest,
                                           double& target) {
  const double p = load1(a.p, a.p_dtype, r.p + v);
  target = weight(p);
  rest = target;
  if (r.rest) rest = a.q ? weight(p - (double)load1(a.q, a.q_dtype, r.q + v)) : v == r.drop ? 0.0 : target;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

__global__ void __launch_bounds__(kThreads) slice_sums_kernel(tb_verify_draft_args a, SliceSum* sums) {
  __shared__ SliceSum part[kThreads / 64];
  const int64_t b = blockIdx.y;
  const Row r = find_row(a, b);
  const int64_t first = (int64_t)blockIdx.x * kVerifySlice;
  const int64_t end = min(first + kVerifySlice, a.vocab);
  double rest = 0.0, target = 0.0;
  for (int64_t v = first + threadIdx.x; v < end; v += kThreads) {
    double x, y;
    weights_at(a, r, v, x, y);
    rest += x;
    target += y;
  }
  rest = wave_sum(rest);
  target = wave_sum(target);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = SliceSum{rest, target};
  __syncthreads();
  if (threadIdx.x == 0) {
    SliceSum s = part[0];
    for (int w = 1; w < kThreads / 64; ++w) {
      s.rest += part[w].rest;
      s.target += part[w].target;
    }
    sums[b * gridDim.x + blockIdx.x] = s;
  }
}

// One wave per sequence: the search is a chain of short steps.
__global__ void __launch_bounds__(64) draw_kernel(tb_verify_draft_args a, const SliceSum* sums, int64_t slices) {
  const int64_t b = blockIdx.x;
  const int lane = threadIdx.x;
  const Row r = find_row(a, b);
  const SliceSum* s = sums + b * slices;

  double rest = 0.0, target = 0.0;
  for (int64_t i = lane; i < slices; i += 64) {
    rest += s[i].rest;
    target += s[i].target;
  }
  rest = wave_sum(rest);
  target = wave_sum(target);
  const bool by_rest = rest > 0.0;
  const double goal = (double)a.u_next[b] * (by_rest ? rest : target);

  // the first slice whose end is past the goal; `before` is the sum before it.
  // If rounding (or u_next >= 1) leaves none, the last slice with weight.
  int64_t slice = -1, last = -1;
  double before = 0.0, last_before = 0.0;
  for (int64_t i0 = 0; i0 < slices && slice < 0; i0 += 64) {
    const int64_t i = i0 + lane;
    const double w = i < slices ? (by_rest ? s[i].rest : s[i].target) : 0.0;
    double up = w;  // inclusive prefix over the lanes
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double t = __shfl_up(up, m);
      if (lane >= m) up += t;
    }
    const uint64_t past = __ballot(w > 0.0 && before + up > goal), some = __ballot(w > 0.0);
    if (some) {
      const int l = 63 - __builtin_clzll(some);
      last = i0 + l;
      last_before = before + __shfl(up - w, l);
    }
    if (past) {
      const int l = __builtin_ctzll(past);
      slice = i0 + l;
      last_before = before + __shfl(up - w, l);
    }
    before += __shfl(up, 63);
  }
  if (slice < 0) slice = last;
  before = last_before;

  int token = -1;
  if (slice >= 0) {
    const int64_t first = slice * kVerifySlice, end = min(first + kVerifySlice, a.vocab);
    int64_t found = -1, fallback = -1;
    for (int64_t v0 = first; v0 < end && found < 0; v0 += 64) {
      const int64_t v = v0 + lane;
      double x = 0.0, y = 0.0;
      if (v < end) weights_at(a, r, v, x, y);
      const double w = by_rest ? x : y;
      double up = w;
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {
        const double t = __shfl_up(up, m);
        if (lane >= m) up += t;
      }
      const uint64_t past = __ballot(w > 0.0 && before + up > goal), some = __ballot(w > 0.0);
      if (some) fallback = v0 + 63 - __builtin_clzll(some);
      if (past) found = v0 + __builtin_ctzll(past);
      before += __shfl(up, 63);
    }
    token = (int)(found >= 0 ? found : fallback);
  }

  if (lane == 0) a.accepted[b] = r.kept;
  for (int j = lane; j <= a.max_draft; j += 64) {
    int t = -1;
    if (j < r.kept) t = a.drafts[r.seq_at + j];
    else if (j == r.kept) t = token;
    a.tokens[b * (a.max_draft + 1) + j] = t;
  }
}

}  // namespace

hipError_t launch_verify_draft(const tb_verify_draft_args& a, hipStream_t stream) {
  const int64_t slices = (a.vocab + kVerifySlice - 1) / kVerifySlice;
  SliceSum* sums = static_cast<SliceSum*>(a.workspace);
  hipLaunchKernelGGL(slice_sums_kernel, dim3((unsigned)slices, (unsigned)a.B), dim3(kThreads), 0, stream, a, sums);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(draw_kernel, dim3((unsigned)a.B), dim3(64), 0, stream, a, sums, slices);
  return hipGetLastError();
}

}  // namespace tb
