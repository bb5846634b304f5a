// Verification of drafted tokens against the target's probabilities, from
// given random numbers (include/tb.h, tb_verify_draft).
//
// What has to be read is one row of p and one of q per sequence: the row where
// the first token is not kept.  Each wave finds it by itself, a gather of at
// most TB_MAX_DRAFT pairs.  The row is cut into slices; with all their sums,
// the slice that holds u_next * sum is read again, four entries a thread, for
// the token.  Up to kVerifyWhole entries the slices are the waves of one
// workgroup, and a sequence takes one launch.  Larger vocabularies have a
// workgroup per slice and a second launch.  The search over the slices is done
// by every wave for itself, so a draw has one barrier.
// Differences and sums are in 64 bits, so that which token an edge falls to
// does not depend on how the sum is split.
//
// Bound by latency: the chain draft - its probabilities - the row - the slice -
// the token (one sequence of 32003 entries: 8.4 us in one launch, 5.5 + 4.6 in
// two), and by HBM where the rows are many (32 of 131073 entries, fp32, 33.6
// MB: 8.7 us for the sums, 3.9 TB/s, and 4.6 for the draw; by one workgroup
// each 30 us, as a CU reads 0.1 TB/s at best).
#include "tb_common.h"
#include "tb_launch.h"
#include "wave_scan.h"

namespace tb {

namespace {

constexpr int kThreads = 256;    // of a slice's sum
constexpr int kDrawWaves = 16;   // of a sequence's draw

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
  int kept;         // drafts that are kept
  int drop;         // certain drafter: the token that is not kept (else -1)
  bool rest;        // weights max(p - q, 0), not p
};

// The row of sequence b when `kept` of its drafts are kept.
__device__ __forceinline__ Row row_of(const tb_verify_draft_args& a, int64_t b, int64_t lo, int T, int kept) {
  Row r;
  r.seq_at = lo;
  r.kept = kept;
  r.rest = kept < T;
  r.p = (lo + b + kept) * a.p_stride;
  r.q = r.rest ? (lo + kept) * a.q_stride : 0;
  r.drop = r.rest && !a.q ? a.drafts[lo + kept] : -1;
  return r;
}

__device__ __forceinline__ int drafts_of(const tb_verify_draft_args& a, int64_t b, int64_t& lo) {
  lo = min(max((int64_t)a.cu_draft[b], (int64_t)0), a.total);
  const int64_t hi = min(max((int64_t)a.cu_draft[b + 1], lo), a.total);
  return (int)min(hi - lo, (int64_t)a.max_draft);
}

// Every lane of the wave calls this with the same b; the same answer in each.
__device__ __forceinline__ Row find_row(const tb_verify_draft_args& a, int64_t b) {
  int64_t lo;
  const int T = drafts_of(a, b, lo), j = threadIdx.x & 63;
  bool keep = false;
  if (j < T) {
    const int d = a.drafts[lo + j];
    if (d >= 0 && d < a.vocab) {
      const double pd = load1(a.p, a.p_dtype, (lo + b + j) * a.p_stride + d);
      const double qd = a.q ? (double)load1(a.q, a.q_dtype, (lo + j) * a.q_stride + d) : 1.0;
      keep = (double)a.u[lo + j] * qd < pd;
    }
  }
  const uint64_t lost = ~__ballot(keep);
  return row_of(a, b, lo, T, lost == 0 ? 64 : __builtin_ctzll(lost));
}

// four consecutive entries; a row starts at any element, so these loads are
// aligned to elements only
template <int DTYPE>
__device__ __forceinline__ void load4(const void* p, int64_t i, float (&v)[4]) {
  if constexpr (DTYPE == TB_BF16) {
    typedef uint16_t __attribute__((ext_vector_type(4), aligned(2))) u16x4;
    const u16x4 w = *reinterpret_cast<const u16x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = bf16_to_f32(w[e]);
  } else {
    typedef float __attribute__((ext_vector_type(4), aligned(4))) f32x4u;
    const f32x4u w = *reinterpret_cast<const f32x4u*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = w[e];
  }
}

// The weights of four entries, and of the first n < 4; QD < 0: no q.
template <int PD, int QD>
__device__ __forceinline__ void weights4(const tb_verify_draft_args& a, const Row& r, int64_t v, int n,
                                         double (&rest)[4], double (&target)[4]) {
  float p[4] = {0.f, 0.f, 0.f, 0.f}, q[4] = {0.f, 0.f, 0.f, 0.f};
  if (n >= 4) {
    load4<PD>(a.p, r.p + v, p);
    if constexpr (QD >= 0) load4<QD>(a.q, r.q + v, q);
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) {
        p[e] = load1(a.p, PD, r.p + v + e);
        if constexpr (QD >= 0) q[e] = load1(a.q, QD, r.q + v + e);
      }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    target[e] = weight(p[e]);
    rest[e] = !r.rest ? target[e] : QD < 0 ? (v + e == r.drop ? 0.0 : target[e]) : weight((double)p[e] - q[e]);
  }
}

// One thread's share of the sum over [begin, end): four entries at 4 * `t`, and
// every 4 * `threads` from there.
template <int PD, int QD>
__device__ __forceinline__ SliceSum sum_share(const tb_verify_draft_args& a, const Row& r, int64_t begin, int64_t end,
                                              int t, int threads) {
  SliceSum s{0.0, 0.0};
  double rest[4], target[4];
  int64_t v = begin + 4 * t;
#pragma unroll 4
  for (; v + 4 <= end; v += 4 * threads) {
    weights4<PD, QD>(a, r, v, 4, rest, target);
    s.rest += (rest[0] + rest[1]) + (rest[2] + rest[3]);
    s.target += (target[0] + target[1]) + (target[2] + target[3]);
  }
  if (v < end) {  // of the one thread whose next four reach past the end
    weights4<PD, QD>(a, r, v, (int)(end - v), rest, target);
    s.rest += rest[0] + rest[1] + rest[2];
    s.target += target[0] + target[1] + target[2];
  }
  return s;
}

// Of the lanes' sums `w` in order, from `before` on: the first lane with weight
// whose end is past the goal.
struct Lane {
  int first, last;  // that lane; the last with weight (-1: none)
  double end;       // the sum up to and with this lane
};
__device__ __forceinline__ Lane find_lane(double w, double before, double goal) {
  Lane l;
  l.end = before + wave_prefix(w);
  const uint64_t past = __ballot(w > 0.0 && l.end > goal), some = __ballot(w > 0.0);
  l.first = past ? __builtin_ctzll(past) : -1;
  l.last = some ? 63 - __builtin_clzll(some) : -1;
  return l;
}

// A sequence's draw by kDrawWaves waves, from the sums of its slices (in order,
// `length` entries each, at most four for a thread), and its answer: the kept
// drafts, the drawn token, then -1.
template <int PD, int QD>
__device__ __forceinline__ void draw(const tb_verify_draft_args& a, int64_t b, const Row& r, double u,
                                     const SliceSum* s, int64_t slices, int length) {
  __shared__ double wave_sums[kDrawWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double rest = 0.0, target = 0.0;
  for (int64_t i = lane; i < slices; i += 64) {
    rest += s[i].rest;
    target += s[i].target;
  }
  rest = wave_sum(rest);
  target = wave_sum(target);
  const bool by_rest = rest > 0.0;
  const double goal = u * (by_rest ? rest : target);

  // the first slice whose end is past the goal; if rounding (or u_next >= 1)
  // leaves none, the last with weight
  int64_t slice = -1;
  double before = 0.0, sum = 0.0;
  for (int64_t i0 = 0; i0 < slices; i0 += 64) {
    const int64_t i = i0 + lane;
    const double w = i < slices ? (by_rest ? s[i].rest : s[i].target) : 0.0;
    const Lane l = find_lane(w, sum, goal);
    const int who = l.first >= 0 ? l.first : l.last;
    if (who >= 0) {
      slice = i0 + who;
      before = of_lane(l.end, who) - of_lane(w, who);
    }
    if (l.first >= 0) break;
    sum = of_lane(l.end, 63);
  }

  // its entries: the same over the waves (by each wave for itself), over the
  // lanes of the one found, and over a lane's four
  int64_t v = 0;
  double w[4] = {0.0, 0.0, 0.0, 0.0};
  if (slice >= 0) {
    const int64_t first = slice * length, end = min(first + length, a.vocab);
    v = first + 4 * (int)threadIdx.x;
    if (v < end) {
      double x[4], y[4];
      weights4<PD, QD>(a, r, v, (int)min(end - v, (int64_t)4), x, y);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = by_rest ? x[e] : y[e];
    }
  }
  const double own = (w[0] + w[1]) + (w[2] + w[3]), mine = wave_sum(own);
  if (lane == 0) wave_sums[wave] = mine;
  __syncthreads();
  const double each = lane < kDrawWaves ? wave_sums[lane] : 0.0;
  const Lane l = find_lane(each, before, goal);
  const int who = l.first >= 0 ? l.first : l.last;
  if (wave != (who < 0 ? 0 : who)) return;

  int token = -1;
  if (who >= 0) {
    const Lane in = find_lane(own, of_lane(l.end, who) - of_lane(each, who), goal);
    const int at = in.first >= 0 ? in.first : in.last;
    double end = in.end - own;
    bool past = false;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (w[e] > 0.0 && !past) {
        token = (int)(v + e);
        end += w[e];
        past = end > goal;
      }
    token = __builtin_amdgcn_readlane(token, at);
  }
  if (lane == 0) a.accepted[b] = r.kept;
  for (int j = lane; j <= a.max_draft; j += 64) {
    int t = -1;
    if (j < r.kept) t = a.drafts[r.seq_at + j];
    else if (j == r.kept) t = token;
    a.tokens[b * (a.max_draft + 1) + j] = t;
  }
}

// One workgroup per sequence, one wave per slice.
template <int PD, int QD>
__global__ void __launch_bounds__(64 * kDrawWaves) whole_kernel(tb_verify_draft_args a) {
  __shared__ SliceSum sums[kDrawWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t b = blockIdx.x;
  const double u = a.u_next[b];
  const Row r = find_row(a, b);
  const int length = (int)((a.vocab + 256 * kDrawWaves - 1) / (256 * kDrawWaves)) * 256;
  const int64_t begin = min((int64_t)wave * length, a.vocab);
  SliceSum s = sum_share<PD, QD>(a, r, begin, min(begin + length, a.vocab), lane, 64);
  s.rest = wave_sum(s.rest);
  s.target = wave_sum(s.target);
  if (lane == 0) sums[wave] = s;
  __syncthreads();
  draw<PD, QD>(a, b, r, u, sums, kDrawWaves, length);
}

// `kept` [B]: for the second launch.
template <int PD, int QD>
__global__ void __launch_bounds__(kThreads) slice_sums_kernel(tb_verify_draft_args a, SliceSum* sums, int* kept) {
  __shared__ SliceSum part[kThreads / 64];
  const int64_t b = blockIdx.y;
  const Row r = find_row(a, b);
  const int64_t begin = (int64_t)blockIdx.x * kVerifySlice;
  SliceSum s = sum_share<PD, QD>(a, r, begin, min(begin + kVerifySlice, a.vocab), threadIdx.x, kThreads);
  s.rest = wave_sum(s.rest);
  s.target = wave_sum(s.target);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = part[0];
    for (int w = 1; w < kThreads / 64; ++w) {
      s.rest += part[w].rest;
      s.target += part[w].target;
    }
    sums[b * gridDim.x + blockIdx.x] = s;
    if (blockIdx.x == 0) kept[b] = r.kept;
  }
}

template <int PD, int QD>
__global__ void __launch_bounds__(64 * kDrawWaves) draw_kernel(tb_verify_draft_args a, const SliceSum* sums,
                                                               const int* kept, int64_t slices) {
  const int64_t b = blockIdx.x;
  const double u = a.u_next[b];
  const int n = kept[b];
  int64_t lo;
  const int T = drafts_of(a, b, lo);
  draw<PD, QD>(a, b, row_of(a, b, lo, T, n), u, sums + b * slices, slices, (int)kVerifySlice);
}

static_assert(kVerifySlice == 4 * 64 * kDrawWaves && kVerifyWhole <= kDrawWaves * kVerifySlice, "four entries a thread");

template <int PD, int QD>
hipError_t launch(const tb_verify_draft_args& a, hipStream_t stream) {
  if (a.vocab <= kVerifyWhole) {
    hipLaunchKernelGGL((whole_kernel<PD, QD>), dim3((unsigned)a.B), dim3(64 * kDrawWaves), 0, stream, a);
    return hipGetLastError();
  }
  const int64_t slices = (a.vocab + kVerifySlice - 1) / kVerifySlice;
  SliceSum* sums = static_cast<SliceSum*>(a.workspace);
  int* kept = reinterpret_cast<int*>(sums + a.B * slices);
  hipLaunchKernelGGL((slice_sums_kernel<PD, QD>), dim3((unsigned)slices, (unsigned)a.B), dim3(kThreads), 0, stream, a,
                     sums, kept);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((draw_kernel<PD, QD>), dim3((unsigned)a.B), dim3(64 * kDrawWaves), 0, stream, a, sums, kept,
                     slices);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_verify_draft(const tb_verify_draft_args& a, hipStream_t stream) {
  const bool pb = a.p_dtype == TB_BF16, qb = a.q_dtype == TB_BF16;
  if (!a.q) return pb ? launch<TB_BF16, -1>(a, stream) : launch<TB_F32, -1>(a, stream);
  if (pb) return qb ? launch<TB_BF16, TB_BF16>(a, stream) : launch<TB_BF16, TB_F32>(a, stream);
  return qb ? launch<TB_F32, TB_BF16>(a, stream) : launch<TB_F32, TB_F32>(a, stream);
}

}  // namespace tb
