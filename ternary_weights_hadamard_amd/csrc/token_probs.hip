// The probabilities of tokens from logits: biases, penalties of repeated tokens,
// grammar masks, temperature and softmax (include/tb.h, tb_token_probs).
//
// What changes a logit is known by its token: for a run of the vocabulary, LDS
// holds a word for each entry (its bias, how often it was generated, whether the
// prompt has it), made from the sequence's lists by integer atomics, so that
// results do not depend on their order.  The lists are read once for all rows of
// a sequence that a workgroup has: from one row to the next a draft is added.
//
// Up to kProbsWhole entries a workgroup has a row in registers: one launch, each
// logit read once.  Larger vocabularies have a workgroup for a slice: the first
// launch leaves each slice's maximum, sum and first maximum, the second reads the
// logits again (from the caches, where they fit) and writes.
#include "tb_common.h"
#include "tb_launch.h"

namespace tb {

namespace {

constexpr int kThreads = 256;   // of a slice
constexpr uint32_t kCount = (1u << 20) - 1, kTold = 1u << 31;
constexpr int kBiasShift = 20;
constexpr float kLog2e = 1.4426950408889634f;
static_assert(TB_MAX_BIAS < (1 << 11) && kProbsSlice == 16 * kThreads, "a word's fields; four loads of four a thread");

// A sequence: its rows, its lists and its parameters.
struct Seq {
  int64_t row0;            // of its first row
  int64_t draft0;
  int drafts;
  int64_t told, made, end;  // its history: the prompt from `told`, generated from `made`
  int64_t bias;
  int biases;
  float sharp;             // log2(e) / temperature; 0: the largest is taken
  float repeats, presence, frequency;
};

struct Range {
  int64_t lo, hi;
};
__device__ __forceinline__ Range range_of(const int32_t* cu, int64_t b, int64_t total) {
  Range r;
  r.lo = min(max((int64_t)cu[b], (int64_t)0), total);
  r.hi = min(max((int64_t)cu[b + 1], r.lo), total);
  return r;
}

__device__ __forceinline__ Seq sequence(const tb_token_probs_args& a, int64_t b) {
  Seq s{};
  if (a.cu_draft) {
    const Range d = range_of(a.cu_draft, b, a.total);
    s.draft0 = d.lo;
    s.drafts = (int)min(d.hi - d.lo, (int64_t)a.max_draft);
  }
  s.row0 = s.draft0 + b;
  if (a.history) {
    const Range h = range_of(a.cu_history, b, a.total_history);
    const int64_t prompt = a.prompt_len ? min(max((int64_t)a.prompt_len[b], (int64_t)0), h.hi - h.lo) : 0;
    s.told = h.lo;
    s.made = h.lo + prompt;
    s.end = h.hi;
  }
  if (a.bias_ids) {
    const Range r = range_of(a.cu_bias, b, a.total_bias);
    s.bias = r.lo;
    s.biases = (int)min(r.hi - r.lo, (int64_t)TB_MAX_BIAS);
  }
  const f32x4 p = *reinterpret_cast<const f32x4*>(a.params + 4 * b);
  s.sharp = p[0] > 0.f ? fminf(fmaxf(kLog2e / p[0], 1.4e-45f), 3e38f) : 0.f;  // no 0 * inf
  s.repeats = p[1];
  s.presence = p[2];
  s.frequency = p[3];
  return s;
}

__device__ __forceinline__ void add_draft(const tb_token_probs_args& a, const Seq& s, int j, uint32_t* words, int64_t begin,
                                          int64_t end) {
  const int64_t id = a.drafts[s.draft0 + j];
  if (id >= begin && id < end) atomicAdd(words + (id - begin), 1u);
}

// The words of entries begin .. end - 1 for a row behind `j` drafts; `count` of
// them are cleared (a multiple of 4 * THREADS).  Barriers before, between and behind.
template <int THREADS>
__device__ __forceinline__ void make_words(const tb_token_probs_args& a, const Seq& s, int j, uint32_t* words, int count,
                                           int64_t begin, int64_t end) {
  const int tid = threadIdx.x;
  for (int i = 4 * tid; i < count; i += 4 * THREADS) *reinterpret_cast<u32x4*>(words + i) = u32x4{0u, 0u, 0u, 0u};
  __syncthreads();
  if (s.biases > 0) {
    for (int i = tid; i < s.biases; i += THREADS) {
      const int64_t id = a.bias_ids[s.bias + i];
      if (id >= begin && id < end) atomicMax(words + (id - begin), (uint32_t)(i + 1) << kBiasShift);
    }
    __syncthreads();  // the words are only biases yet: the last one of an id is the largest
  }
  // no more than the count has room for, with all drafts
  const int64_t counted = max(s.made, s.end - ((1 << 20) - TB_MAX_DRAFT));
#pragma unroll 4
  for (int64_t i = s.told + tid; i < s.end; i += THREADS) {
    const int64_t id = a.history[i];
    if (id < begin || id >= end) continue;
    if (i < s.made) atomicOr(words + (id - begin), kTold);
    else if (i >= counted) atomicAdd(words + (id - begin), 1u);
  }
  if (tid < j) add_draft(a, s, tid, words, begin, end);
  __syncthreads();
}

__device__ __forceinline__ float adjusted(const tb_token_probs_args& a, const Seq& s, float x, uint32_t word) {
  const uint32_t bias = word >> kBiasShift & 0x7ffu, count = word & kCount;
  if (bias) x += a.bias_values[s.bias + bias - 1];
  if (word & (kTold | kCount)) x = x > 0.f ? x / s.repeats : x * s.repeats;
  if (count) x -= s.frequency * (float)count + s.presence;
  return x;
}

template <int DTYPE>
__device__ __forceinline__ f32x4 load4(const void* p, int64_t i, int n) {
  f32x4 v = {-__builtin_inff(), -__builtin_inff(), -__builtin_inff(), -__builtin_inff()};
  if constexpr (DTYPE == TB_BF16) {
    typedef uint16_t __attribute__((ext_vector_type(4), aligned(2))) u16x4;
    const uint16_t* from = static_cast<const uint16_t*>(p) + i;
    if (n >= 4) {
      const u16x4 w = *reinterpret_cast<const u16x4*>(from);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = bf16_to_f32(w[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) v[e] = bf16_to_f32(from[e]);
    }
  } else {
    typedef float __attribute__((ext_vector_type(4), aligned(4))) f32x4u;
    const float* from = static_cast<const float*>(p) + i;
    if (n >= 4) {
      const f32x4u w = *reinterpret_cast<const f32x4u*>(from);
      v = f32x4{w[0], w[1], w[2], w[3]};
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) v[e] = from[e];
    }
  }
  return v;
}

template <int DTYPE>
__device__ __forceinline__ void store4(void* p, int64_t i, int n, const f32x4& v) {
  if constexpr (DTYPE == TB_BF16) {
    typedef uint16_t __attribute__((ext_vector_type(4), aligned(2))) u16x4;
    uint16_t* to = static_cast<uint16_t*>(p) + i;
    u16x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = (uint16_t)f32_to_bf16_rne(v[e]);
    if (n >= 4) {
      *reinterpret_cast<u16x4*>(to) = w;
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) to[e] = w[e];
    }
  } else {
    typedef float __attribute__((ext_vector_type(4), aligned(4))) f32x4u;
    float* to = static_cast<float*>(p) + i;
    if (n >= 4) {
      *reinterpret_cast<f32x4u*>(to) = f32x4u{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) to[e] = v[e];
    }
  }
}

// The row's mask, or NULL.
__device__ __forceinline__ const uint32_t* mask_of(const tb_token_probs_args& a, int64_t row) {
  if (!a.mask) return nullptr;
  const int64_t m = a.mask_row ? (int64_t)a.mask_row[row] : row;
  return m >= 0 && m < a.n_masks ? a.mask + m * a.mask_stride : nullptr;
}

// A thread's entries of a row: 4 at v0 + CHUNK * c for each c, as loaded, and
// what the formula makes of them; past the end of the row -inf.
template <int CHUNKS, int CHUNK, int LD>
struct Mine {
  f32x4 x[CHUNKS];
  uint32_t allowed[CHUNKS];  // from bit 0 on
  __device__ __forceinline__ void load(const tb_token_probs_args& a, int64_t row, int64_t v0) {
    const uint32_t* mask = mask_of(a, row);
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int64_t v = v0 + CHUNK * c, n = a.vocab - v;
      x[c] = f32x4{-__builtin_inff(), -__builtin_inff(), -__builtin_inff(), -__builtin_inff()};
      allowed[c] = 0xfu;
      if (n <= 0) continue;
      x[c] = load4<LD>(a.logits, row * a.logits_stride + v, (int)min(n, (int64_t)4));
      if (mask) allowed[c] = mask[v >> 5] >> (v & 31);  // v is a multiple of 4
    }
  }
  // `words` of the thread's first entry
  template <bool WORDS>
  __device__ __forceinline__ void adjust(const tb_token_probs_args& a, const Seq& s, const uint32_t* words) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      u32x4 w = {0u, 0u, 0u, 0u};
      if constexpr (WORDS) w = *reinterpret_cast<const u32x4*>(words + CHUNK * c);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (WORDS && w[e]) x[c][e] = adjusted(a, s, x[c][e], w[e]);
        if (!((allowed[c] >> e) & 1u)) x[c][e] = -__builtin_inff();
      }
    }
  }
  __device__ __forceinline__ float top() const {
    float m = -__builtin_inff();
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = fmaxf(m, x[c][e]);
    return m;
  }
  // the first entry that is `m`
  __device__ __forceinline__ int first(int64_t v0, float m) const {
    int at = INT32_MAX;
#pragma unroll
    for (int c = CHUNKS - 1; c >= 0; --c)
#pragma unroll
      for (int e = 3; e >= 0; --e)
        if (x[c][e] == m) at = (int)(v0 + CHUNK * c + e);
    return m == -__builtin_inff() ? INT32_MAX : at;
  }
  // turned into weights relative to m (not -inf), and their sum
  __device__ __forceinline__ float weigh(float m, float sharp) {
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[c][e] = __builtin_amdgcn_exp2f((x[c][e] - m) * sharp);
      sum += (x[c][0] + x[c][1]) + (x[c][2] + x[c][3]);
    }
    return sum;
  }
  template <int PD>
  __device__ __forceinline__ void write(const tb_token_probs_args& a, int64_t row, int64_t v0, float f, int hot) const {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int64_t v = v0 + CHUNK * c, n = a.vocab - v;
      if (n <= 0) continue;
      f32x4 p;
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = hot >= 0 ? (v + e == hot ? 1.f : 0.f) : x[c][e] * f;
      store4<PD>(a.p, row * a.p_stride + v, (int)min(n, (int64_t)4), p);
    }
  }
};

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}
__device__ __forceinline__ float wave_add(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}
__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = min(v, __shfl_xor(v, m));
  return v;
}

// Over the WAVES waves of the workgroup, in a fixed order; a barrier.  Between
// two calls with the same array there has to be another.
template <int WAVES, typename T, typename J>
__device__ __forceinline__ T over_waves(T v, T* of_wave, J join) {
  of_wave[threadIdx.x >> 6] = v;
  __syncthreads();
  v = of_wave[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) v = join(v, of_wave[w]);
  return v;
}

constexpr float kNone = -__builtin_inff();

// One workgroup a row, of CHUNKS * 4096 entries at most.
template <int LD, int PD, int CHUNKS, bool WORDS>
__global__ void __launch_bounds__(1024) whole_kernel(tb_token_probs_args a) {
  constexpr int kWaves = 16, kChunk = 4096;
  __shared__ __align__(16) uint32_t words[WORDS ? CHUNKS * kChunk : 4];
  __shared__ float tops[kWaves], sums[kWaves];
  __shared__ int firsts[kWaves];
  const int64_t b = blockIdx.y;
  const int j = blockIdx.x;
  const Seq s = sequence(a, b);
  if (j > s.drafts) return;
  const int64_t row = s.row0 + j, v0 = 4 * (int)threadIdx.x;
  Mine<CHUNKS, kChunk, LD> mine;
  mine.load(a, row, v0);
  if constexpr (WORDS) make_words<1024>(a, s, j, words, CHUNKS * kChunk, 0, a.vocab);
  mine.template adjust<WORDS>(a, s, words + v0);
  const float m = over_waves<kWaves>(wave_max(mine.top()), tops, [](float x, float y) { return fmaxf(x, y); });
  int hot = -1;
  float f = 0.f;
  if (s.sharp > 0.f) {
    const float sum = mine.weigh(m == kNone ? 0.f : m, s.sharp);
    const float total = over_waves<kWaves>(wave_add(sum), sums, [](float x, float y) { return x + y; });
    f = total == 0.f ? 0.f : 1.f / total;
  } else {
    hot = over_waves<kWaves>(wave_min(mine.first(v0, m)), firsts, [](int x, int y) { return min(x, y); });
  }
  mine.template write<PD>(a, row, v0, f, hot);
}

// What a slice leaves for its row.
struct Slice {
  float top, sum;  // the weights' sum relative to the top
  int first;       // the first entry at the top
  int reserved;
};

// Rows part * per .. of a sequence, over one slice of the vocabulary.
template <int LD, int PD, bool WORDS, bool WRITE>
__global__ void __launch_bounds__(kThreads) slice_kernel(tb_token_probs_args a, Slice* slices, int per) {
  constexpr int kWaves = kThreads / 64, kChunk = 4 * kThreads, kChunks = kProbsSlice / kChunk;
  __shared__ __align__(16) uint32_t words[WORDS ? kProbsSlice : 4];
  __shared__ float tops[kWaves], sums[kWaves];
  __shared__ int firsts[kWaves];
  const int64_t b = blockIdx.y, begin = (int64_t)blockIdx.x * kProbsSlice, v0 = begin + 4 * (int)threadIdx.x;
  const Seq s = sequence(a, b);
  int j = blockIdx.z * per;
  const int last = min(j + per - 1, s.drafts);
  if (j > last) return;
  Mine<kChunks, kChunk, LD> mine;
  mine.load(a, s.row0 + j, v0);
  const int64_t end = min(begin + kProbsSlice, a.vocab);
  if constexpr (WORDS) make_words<kThreads>(a, s, j, words, kProbsSlice, begin, end);
  for (;; ++j) {
    const int64_t row = s.row0 + j;
    mine.template adjust<WORDS>(a, s, words + (v0 - begin));
    Slice* of_row = slices + row * gridDim.x;
    if constexpr (WRITE) {
      // all slices of the row, by every wave for itself
      Slice all{kNone, 0.f, INT32_MAX, 0};
      for (int64_t i = threadIdx.x & 63; i < gridDim.x; i += 64) {
        const Slice x = of_row[i];
        const float m = fmaxf(all.top, x.top), base = m == kNone ? 0.f : m;
        all.sum = all.sum * __builtin_amdgcn_exp2f((all.top - base) * s.sharp) +
                  x.sum * __builtin_amdgcn_exp2f((x.top - base) * s.sharp);
        if (x.top > all.top) all.first = x.first;  // slices come in order
        all.top = m;
      }
      const float m = wave_max(all.top), base = m == kNone ? 0.f : m;
      if (s.sharp > 0.f) {
        const float total = wave_add(all.sum * __builtin_amdgcn_exp2f((all.top - base) * s.sharp));
        mine.weigh(base, s.sharp);
        mine.template write<PD>(a, row, v0, total == 0.f ? 0.f : 1.f / total, -1);
      } else {
        const int hot = wave_min(all.top == m ? all.first : INT32_MAX);
        mine.template write<PD>(a, row, v0, 0.f, hot);
      }
    } else {
      const float m = over_waves<kWaves>(wave_max(mine.top()), tops, [](float x, float y) { return fmaxf(x, y); });
      Slice out{m, 0.f, INT32_MAX, 0};
      if (s.sharp > 0.f) {
        const float sum = mine.weigh(m == kNone ? 0.f : m, s.sharp);
        out.sum = over_waves<kWaves>(wave_add(sum), sums, [](float x, float y) { return x + y; });
      } else {
        out.first = over_waves<kWaves>(wave_min(mine.first(v0, m)), firsts, [](int x, int y) { return min(x, y); });
      }
      if (threadIdx.x == 0) of_row[blockIdx.x] = out;
    }
    if (j == last) return;
    mine.load(a, row + 1, v0);
    if constexpr (WORDS) {
      __syncthreads();
      if (threadIdx.x == 0) add_draft(a, s, j, words, begin, end);
      __syncthreads();
    }
  }
}

template <int LD, int PD, bool WORDS>
hipError_t launch(const tb_token_probs_args& a, hipStream_t stream) {
  if (a.vocab <= kProbsWhole) {
    const dim3 grid((unsigned)a.max_draft + 1, (unsigned)a.B), block(1024);
    if (a.vocab <= 4096) hipLaunchKernelGGL((whole_kernel<LD, PD, 1, WORDS>), grid, block, 0, stream, a);
    else if (a.vocab <= 8192) hipLaunchKernelGGL((whole_kernel<LD, PD, 2, WORDS>), grid, block, 0, stream, a);
    else if (a.vocab <= 16384) hipLaunchKernelGGL((whole_kernel<LD, PD, 4, WORDS>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((whole_kernel<LD, PD, 8, WORDS>), grid, block, 0, stream, a);
    return hipGetLastError();
  }
  // Rows of a sequence share a workgroup, so that its lists are read once for
  // them, but not so many that fewer than four workgroups are left for a CU.
  const int64_t slices = (a.vocab + kProbsSlice - 1) / kProbsSlice, rows = a.max_draft + 1;
  int64_t parts = (1024 + slices * a.B - 1) / (slices * a.B);
  if (parts > rows) parts = rows;
  const int per = (int)((rows + parts - 1) / parts);
  const dim3 grid((unsigned)slices, (unsigned)a.B, (unsigned)((rows + per - 1) / per)), block(kThreads);
  Slice* of = static_cast<Slice*>(a.workspace);
  hipLaunchKernelGGL((slice_kernel<LD, PD, WORDS, false>), grid, block, 0, stream, a, of, per);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((slice_kernel<LD, PD, WORDS, true>), grid, block, 0, stream, a, of, per);
  return hipGetLastError();
}

template <int LD, int PD>
hipError_t launch(const tb_token_probs_args& a, hipStream_t stream) {
  const bool words = a.history || a.bias_ids || a.total > 0;
  return words ? launch<LD, PD, true>(a, stream) : launch<LD, PD, false>(a, stream);
}

}  // namespace

static_assert(sizeof(Slice) == kProbsSliceBytes, "the workspace's size");

hipError_t launch_token_probs(const tb_token_probs_args& a, hipStream_t stream) {
  const bool lb = a.logits_dtype == TB_BF16, pb = a.p_dtype == TB_BF16;
  if (lb) return pb ? launch<TB_BF16, TB_BF16>(a, stream) : launch<TB_BF16, TB_F32>(a, stream);
  return pb ? launch<TB_F32, TB_BF16>(a, stream) : launch<TB_F32, TB_F32>(a, stream);
}

}  // namespace tb
