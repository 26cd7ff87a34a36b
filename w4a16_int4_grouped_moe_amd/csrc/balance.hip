// balance.hip -- the router's balance loss, its counts and its gradient (gfx950).
//
// A wave takes tokens one after the other, lane l the experts l, l + 64, ...: softmax with
// its maximum and sum over the wave, p added up in registers. A work-group's waves
// add theirs in fp64 into a piece (one for each sequence that its tokens are in);
// its ids are counted in LDS, by integer atomics, whose order changes nothing. A
// second launch adds the pieces of a sequence in their order, a third one the
// sequences; a batch of one piece is finished by the work-group itself. The
// gradient is one more pass over the scores:
//   p_te (c_be - sum_f c_bf p_tf), with c less its mean k n / S: sum_f p_tf = 1, and
// counts near each other then lose nothing in the difference.
//
// 32768 tokens of 384 experts in 24 sequences (50 MB of scores): 17.8 us for the pieces, 2.8 TB/s, a
// wave waiting in 64% of its cycles, of which about 7 us are a work-group's own start, counts and
// sums (64 tokens, one work-group, take 7.8 us); 3.9 and 2.1 us for the two launches after it;
// 21.3 us for the gradient, 4.7 TB/s. More work-groups of half the size, or the next tokens' scores
// asked for ahead, took as long.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe_balance.h"
#include "balance_internal.h"

namespace balance {
namespace {

template <int TYPE>
struct Score;
template <>
struct Score<MOE_TYPE_FP32> {
  typedef float type;
};
template <>
struct Score<MOE_TYPE_FP16> {
  typedef _Float16 type;
};
template <>
struct Score<MOE_TYPE_BF16> {
  typedef __bf16 type;
};

// x moved across lanes by a DPP control; lanes without a source, or outside
// ROW_MASK, read `none`
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp(float none, float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, x),
                                         CTRL, ROW_MASK, 0xF, false));
}
// op over the wave in a fixed order, returned to every lane
template <typename Op>
__device__ __forceinline__ float wave_reduce(float v, float none, Op op) {
  v = op(v, dpp<0x111, 0xF>(none, v));  // row_shr:1
  v = op(v, dpp<0x112, 0xF>(none, v));  // row_shr:2
  v = op(v, dpp<0x114, 0xF>(none, v));  // row_shr:4
  v = op(v, dpp<0x118, 0xF>(none, v));  // row_shr:8: lane 15 of each row holds the row
  v = op(v, dpp<0x142, 0xA>(none, v));  // row_bcast:15 into rows 1 and 3
  v = op(v, dpp<0x143, 0xC>(none, v));  // row_bcast:31 into rows 2 and 3: lane 63 holds all
  return __builtin_bit_cast(float,
                            __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Row t of a matrix of S values as a resource (t the same for the wave): accesses past it read
// zero and write nothing, so that the kernels need no branches
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_of(const void* matrix, int64_t t, int S) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)((const T*)matrix + t * S), 0,
                                           S * (int)sizeof(T), 0x00020000);
}
// The scores of token t in a lane's registers; experts past S: -inf
template <int NI, typename T>
__device__ __forceinline__ void load_scores(const void* scores, int64_t t, int S, int lane,
                                            float (&v)[NI]) {
  const __amdgpu_buffer_rsrc_t row = row_of<T>(scores, t, S);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 64 * i;
    float x;
    if constexpr (sizeof(T) == 4)
      x = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(row, 4 * e, 0, 0));
    else
      x = (float)__builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(row, 2 * e, 0, 0));
    v[i] = e < S ? x : -__builtin_inff();
  }
}
template <int NI, typename T>
__device__ __forceinline__ void store_scores(void* scores, int64_t t, int S, int lane,
                                             const float (&v)[NI]) {
  const __amdgpu_buffer_rsrc_t row = row_of<T>(scores, t, S);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 64 * i;
    if constexpr (sizeof(T) == 4)
      __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v[i]), row, 4 * e, 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (T)v[i]), row, 2 * e, 0, 0);
  }
}

// v: scores -> softmax. All of them -inf: zeros; +inf and NaN: NaN.
template <int NI>
__device__ __forceinline__ void softmax(float (&v)[NI]) {
  float top = v[0];
#pragma unroll
  for (int i = 1; i < NI; ++i) top = fmaxf(top, v[i]);
  top = wave_reduce(top, -__builtin_inff(), [](float a, float b) { return fmaxf(a, b); });
  if (top == -__builtin_inff()) top = 0.f;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    v[i] = expf(v[i] - top);
    sum += v[i];
  }
  sum = wave_reduce(sum, 0.f, [](float a, float b) { return a + b; });
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < NI; ++i) v[i] *= inv;
}

// The sequence that holds token t: the last b with offsets[b] <= t (-1: none). The whole wave
// looks at 64 offsets at a time: one trip to memory for up to 63 sequences.
__device__ __forceinline__ int sequence_of(const int32_t* __restrict__ offsets, int B, int64_t t,
                                           int lane) {
  int first = 0, n = B + 1;
  for (;;) {
    const int step = (n + 63) / 64;
    const int at = lane * step;
    const int c = __popcll(__ballot(at < n && offsets[first + (at < n ? at : 0)] <= t));
    if (c == 0) return first - 1;
    first += (c - 1) * step;
    n = n - (c - 1) * step < step ? n - (c - 1) * step : step;
    if (step == 1) return first;
  }
}

struct Forward {
  const void* scores;
  const int32_t* ids;
  const uint8_t* mask;
  const int32_t* offsets;
  double* sums;
  int32_t* piece_counts;
  double* parts;
  float* loss;
  int32_t* counts;
  int32_t* tokens;
  int64_t T, per;  // per: tokens of a work-group
  int32_t S, k, B, columns;
};

constexpr int kThreads = 64 * kWaves;

// ALONE: the one work-group of a batch of one sequence ends the loss itself
template <int TYPE, int NI, bool ALONE>
__global__ __launch_bounds__(kThreads) void pieces_kernel(const Forward f) {
  typedef typename Score<TYPE>::type T;
  __shared__ float sums[kWaves][64 * NI];
  __shared__ int32_t hist[64 * NI + 1];
  __shared__ double all[ALONE ? 64 * NI : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t first = (int64_t)blockIdx.x * f.per;
  const int64_t last = first + f.per < f.T ? first + f.per : f.T;
  const int S = f.S;
  int b0 = 0, b1 = 0;
  if (f.offsets) {
    b0 = sequence_of(f.offsets, f.B, first, lane);
    b1 = sequence_of(f.offsets, f.B, last - 1, lane);
    if (b0 < 0) b0 = 0;
    if (b1 >= f.B) b1 = f.B - 1;
  }
  for (int b = b0; b <= b1; ++b) {
    int64_t lo = first, hi = last;
    if (f.offsets) {
      if (f.offsets[b] > lo) lo = f.offsets[b];
      if (f.offsets[b + 1] < hi) hi = f.offsets[b + 1];
      if (lo >= hi) continue;  // the same for every thread
    }
    for (int i = threadIdx.x; i <= S; i += kThreads) hist[i] = 0;
    __syncthreads();
    float acc[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[i] = 0.f;
    for (int64_t t = lo + wave; t < hi; t += kWaves) {
      if (f.mask && !f.mask[t]) continue;
      float v[NI];
      load_scores<NI, T>(f.scores, t, S, lane, v);
      for (int j = lane; j < f.k; j += 64) {
        const int32_t e = f.ids[t * f.k + j];
        if ((uint32_t)e < (uint32_t)S) atomicAdd(&hist[e], 1);
      }
      if (lane == 0) atomicAdd(&hist[S], 1);
      softmax(v);
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[i] += v[i];
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) sums[wave][lane + 64 * i] = acc[i];
    __syncthreads();
    const int64_t piece = (int64_t)blockIdx.x + b;
    for (int e = threadIdx.x; e <= S; e += kThreads) {
      if constexpr (ALONE) {
        if (e < S)
          f.counts[e] = hist[e];
        else
          f.tokens[0] = hist[e];
      } else {
        f.piece_counts[piece * (S + 1) + e] = hist[e];
      }
      if (e == S) continue;
      double s = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) s += sums[w][e];
      if constexpr (ALONE)
        all[e] = s * hist[e];
      else
        f.sums[piece * S + e] = s;
    }
    __syncthreads();
    if constexpr (ALONE) {
      if (wave == 0) {
        double s = 0;
        for (int e = lane; e < S; e += 64) s += all[e];
        for (int x = 32; x; x >>= 1) s += __shfl_xor(s, x);
        const double n = hist[S];
        if (lane == 0) *f.loss = n > 0 ? (float)(s * S / (f.k * n * n)) : 0.f;
      }
    }
  }
  // a sequence's tokens begin after this work-group's only one, or end before it
  if constexpr (ALONE) {
    int64_t lo = 0, hi = f.T;
    if (f.offsets) {
      if (f.offsets[0] > lo) lo = f.offsets[0];
      if (f.offsets[1] < hi) hi = f.offsets[1];
    }
    if (b0 > b1 || lo >= hi) {
      for (int e = threadIdx.x; e < S; e += kThreads) f.counts[e] = 0;
      if (threadIdx.x == 0) *f.loss = 0.f, f.tokens[0] = 0;
    }
  }
}

// One sequence's pieces for 64 experts: counts, tokens and sum_e c_e sum_t p_te.
__global__ __launch_bounds__(kThreads) void sequences_kernel(const Forward f) {
  __shared__ double sums[kWaves][64];
  __shared__ int32_t counts[kWaves][64];
  __shared__ int32_t number[kWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x, S = f.S, e = blockIdx.y * 64 + lane;
  int64_t lo = 0, hi = f.T;
  if (f.offsets) {
    if (f.offsets[b] > lo) lo = f.offsets[b];
    if (f.offsets[b + 1] < hi) hi = f.offsets[b + 1];
  }
  double s = 0;
  int32_t c = 0, n = 0;
  if (lo < hi) {
    const int64_t g1 = (hi - 1) / f.per;
    for (int64_t g = lo / f.per + wave; g <= g1; g += kWaves) {
      const int64_t piece = g + b;
      if (e < S) {
        s += f.sums[piece * S + e];
        c += f.piece_counts[piece * (S + 1) + e];
      }
      n += f.piece_counts[piece * (S + 1) + S];
    }
  }
  sums[wave][lane] = s;
  counts[wave][lane] = c;
  if (lane == 0) number[wave] = n;
  __syncthreads();
  if (wave != 0) return;
  for (int w = 1; w < kWaves; ++w) s += sums[w][lane], c += counts[w][lane], n += number[w];
  if (e < S) f.counts[(int64_t)b * S + e] = c;
  if (blockIdx.y == 0 && lane == 0) f.tokens[b] = n;
  s = e < S ? s * c : 0;
  for (int x = 32; x; x >>= 1) s += __shfl_xor(s, x);
  if (lane == 0) f.parts[(int64_t)b * f.columns + blockIdx.y] = n > 0 ? s / ((double)n * n) : 0;
}

__global__ __launch_bounds__(kThreads) void loss_kernel(const Forward f) {
  __shared__ double sums[kWaves];
  __shared__ int32_t live[kWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  double s = 0;
  int32_t n = 0;
  for (int64_t i = threadIdx.x; i < (int64_t)f.B * f.columns; i += kThreads) s += f.parts[i];
  for (int b = threadIdx.x; b < f.B; b += kThreads) n += f.tokens[b] > 0;
  for (int x = 32; x; x >>= 1) s += __shfl_xor(s, x), n += __shfl_xor(n, x);
  if (lane == 0) sums[wave] = s, live[wave] = n;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kWaves; ++w) s += sums[w], n += live[w];
  *f.loss = n > 0 ? (float)(s * f.S / ((double)f.k * n)) : 0.f;
}

struct Backward {
  const float* dloss;
  const void* scores;
  const int32_t* counts;
  const int32_t* tokens;
  const uint8_t* mask;
  const int32_t* offsets;
  void* dscores;
  int64_t T, per;  // per: tokens of a work-group
  int32_t S, k, B;
};

constexpr int kBackWaves = 4;

template <int TYPE, int NI>
__global__ __launch_bounds__(64 * kBackWaves) void gradient_kernel(const Backward f) {
  typedef typename Score<TYPE>::type T;
  __shared__ int32_t live[kBackWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int S = f.S;
  int n = 0;
  for (int b = threadIdx.x; b < f.B; b += 64 * kBackWaves) n += f.tokens[b] > 0;
  for (int x = 32; x; x >>= 1) n += __shfl_xor(n, x);
  if (lane == 0) live[wave] = n;
  __syncthreads();
  n = live[0] + live[1] + live[2] + live[3];
  const double scale = n > 0 ? (double)*f.dloss * S / ((double)f.k * n) : 0;

  const int64_t first = (int64_t)blockIdx.x * f.per;
  const int64_t last = first + f.per < f.T ? first + f.per : f.T;
  int at = -1, loaded = -1;  // the token's sequence, and the one whose counts are in registers
  int64_t end = -1;          // where the sequence at `at` ends
  float c[NI], factor = 0.f;
  for (int64_t t = first + wave; t < last; t += kBackWaves) {
    float v[NI];
    load_scores<NI, T>(f.scores, t, S, lane, v);  // also of tokens that take no part
    if (t >= end) {
      at = 0, end = f.T;
      if (f.offsets) {
        at = sequence_of(f.offsets, f.B, t, lane);
        if (at >= f.B) at = -1;
        end = at < 0 ? t + 1 : f.offsets[at + 1];
      }
    }
    if (at < 0 || (f.mask && !f.mask[t])) {
#pragma unroll
      for (int i = 0; i < NI; ++i) v[i] = 0.f;
      store_scores<NI, T>(f.dscores, t, S, lane, v);
      continue;
    }
    if (at != loaded) {
      const int32_t tokens = f.tokens[at];
      const int32_t mean = (int32_t)((int64_t)tokens * f.k / S);
#pragma unroll
      for (int i = 0; i < NI; ++i)
        c[i] = lane + 64 * i < S ? (float)(f.counts[(int64_t)at * S + lane + 64 * i] - mean) : 0.f;
      factor = (float)(scale / ((double)tokens * tokens));
      loaded = at;
    }
    softmax(v);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) dot += v[i] * c[i];
    dot = wave_reduce(dot, 0.f, [](float a, float b) { return a + b; });
#pragma unroll
    for (int i = 0; i < NI; ++i) v[i] *= factor * (c[i] - dot);
    store_scores<NI, T>(f.dscores, t, S, lane, v);
  }
}

template <int TYPE, int NI>
void forward_pieces(const Forward& f, bool alone, unsigned groups, hipStream_t stream) {
  if (alone)
    hipLaunchKernelGGL((pieces_kernel<TYPE, NI, true>), dim3(1), dim3(kThreads), 0, stream, f);
  else
    hipLaunchKernelGGL((pieces_kernel<TYPE, NI, false>), dim3(groups), dim3(kThreads), 0, stream,
                       f);
}

// f(an instance of the registers of a lane for S experts)
template <typename F>
void with_registers(int32_t S, F&& f) {
  const int n = (S + 63) / 64;
  if (n <= 1) return f(std::integral_constant<int, 1>{});
  if (n <= 2) return f(std::integral_constant<int, 2>{});
  if (n <= 4) return f(std::integral_constant<int, 4>{});
  if (n <= 6) return f(std::integral_constant<int, 6>{});
  if (n <= 8) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}
template <typename F>
void with_type(int32_t type, F&& f) {
  if (type == MOE_TYPE_BF16) return f(std::integral_constant<int, MOE_TYPE_BF16>{});
  if (type == MOE_TYPE_FP16) return f(std::integral_constant<int, MOE_TYPE_FP16>{});
  return f(std::integral_constant<int, MOE_TYPE_FP32>{});
}

}  // namespace

hipError_t launch_forward(const Sizes& z, const void* scores, const int32_t* ids,
                          const uint8_t* mask, const int32_t* offsets, float* loss,
                          int32_t* counts, int32_t* tokens, void* workspace, hipStream_t stream) {
  const Workspace w(z);
  char* ws = (char*)workspace;
  Forward f{scores, ids, mask, offsets, (double*)(ws + w.sums), (int32_t*)(ws + w.counts),
            (double*)(ws + w.parts), loss, counts, tokens, z.T, group_tokens(z.T), z.S, z.k, z.B,
            column_groups(z.S)};
  if (z.T > 0) {
    const unsigned n = (unsigned)groups(z.T);
    with_type(z.type, [&](auto type) {
      with_registers(z.S, [&](auto ni) {
        forward_pieces<decltype(type)::value, decltype(ni)::value>(f, alone(z), n, stream);
      });
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || alone(z)) return e;
  }
  hipLaunchKernelGGL(sequences_kernel, dim3(z.B, f.columns), dim3(kThreads), 0, stream, f);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(loss_kernel, dim3(1), dim3(kThreads), 0, stream, f);
  return hipGetLastError();
}

hipError_t launch_backward(const Sizes& z, const float* dloss, const void* scores,
                           const int32_t* counts, const int32_t* tokens, const uint8_t* mask,
                           const int32_t* offsets, void* dscores, hipStream_t stream) {
  if (z.T == 0) return hipSuccess;
  // one token a wave until 2048 work-groups, then up to 16, then 2^22 work-groups
  const int64_t fair = (z.T + 2048 * kBackWaves - 1) / (2048 * kBackWaves);
  const int64_t least = (z.T + ((int64_t)kBackWaves << 22) - 1) / ((int64_t)kBackWaves << 22);
  const int64_t per = std::max(std::min<int64_t>(16, fair), least) * kBackWaves;
  const Backward f{dloss, scores, counts, tokens, mask, offsets, dscores, z.T, per, z.S, z.k, z.B};
  const unsigned n = (unsigned)((z.T + per - 1) / per);
  with_type(z.type, [&](auto type) {
    with_registers(z.S, [&](auto ni) {
      hipLaunchKernelGGL((gradient_kernel<decltype(type)::value, decltype(ni)::value>), dim3(n),
                         dim3(64 * kBackWaves), 0, stream, f);
    });
  });
  return hipGetLastError();
}

}  // namespace balance
