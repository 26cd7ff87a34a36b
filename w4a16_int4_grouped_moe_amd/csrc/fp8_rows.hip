// fp8_rows.hip -- the products for a few rows, and the experts' buckets of a few
// (gfx950): decoding, where the time is the weights' way from memory.
//
// A work-group owns 16 weight rows (kSwiglu: 8 gate rows and their 8 up rows) and
// all rows of A, 16 at most; of the experts' short rows several such slices, so that a
// quantised A serves longer streams. Its eight waves take the
// stages of K (128 bytes of a row, one block of scales) in turn. A wave copies its stage's rows into
// LDS in whole 128-byte lines, kD stages ahead, into a place of its own: it waits
// for its own copies alone and never for another wave. At the end the waves'
// sums are added in LDS, in wave order.
//
// A is codes, read straight into the MFMA's layout; or bf16 (or the experts' fp32 h),
// quantised by the work-group into LDS: its first loads go out ahead of the ring's.
// Every work-group repeats it.
//
// Bound by memory and by how long a launch takes to fill and drain it: one token against 4096 x
// 7168 (29 MB) 8.9 us, 3.3 TB/s, a wave waiting in 51% of its cycles; one token's eight experts at
// 7168/2048, 235 MB in 42.8 us (5.5 TB/s) and 117 MB in 23.3 us (5.0 TB/s), waiting in 58 to 60%.
// There three stages in flight and two work-groups on a CU (51 us with four and one), and several
// slices a work-group for the short rows of the second (30 us with one).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "fp8_device.h"
#include "fp8_internal.h"

namespace fp8 {
namespace {

constexpr int kWaves = kRowsWaves, kThreads = 64 * kWaves;
constexpr int kSlot = kRowsSlot;

template <Source SRC, Epilogue EPI, int kD>
__global__ __launch_bounds__(kThreads, 4) void rows_kernel(Product p, const int slices) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr bool kPaired = EPI == kSwiglu, kExperts = EPI == kSwiglu || EPI == kPairs;
  constexpr bool kFresh = SRC != kCodes;
  // an object a stage: the compiler then sees which copies a read has to wait for
  __shared__ __attribute__((aligned(1024))) uint8_t ring0[kWaves * kSlot], ring1[kWaves * kSlot];
  __shared__ __attribute__((aligned(1024))) uint8_t ring2[kWaves * kSlot];
  __shared__ __attribute__((aligned(1024))) uint8_t ring3[kD > 3 ? kWaves * kSlot : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t ring4[kD > 4 ? kWaves * kSlot : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t ring5[kD > 5 ? kWaves * kSlot : 16];
  const lds_bytes ring[6] = {(lds_bytes)ring0, (lds_bytes)ring1, (lds_bytes)ring2,
                             (lds_bytes)ring3, (lds_bytes)ring4, (lds_bytes)ring5};
  // quantised A, then A's scales [row][stage] and B's (kSwiglu: gate, up) [stage]
  extern __shared__ __attribute__((aligned(16))) uint8_t qa[];
  static_assert(kD >= 3 && kD <= 6, "ring objects");

  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int K = (int)p.K, stages = (K + kRow - 1) / kRow;
  constexpr int kStep = rows_step(EPI);  // columns of a slice
  const int N = p.N, n0 = blockIdx.x * kStep * slices;
  const int b_rows = kPaired ? 2 * N : N;
  int M = (int)p.M;
  int64_t first = 0;  // experts: the bucket's first row
  if constexpr (kExperts) {
    first = (int64_t)blockIdx.y * kFewRows;
    if (first >= *p.n_padded) return;  // the grid is sized for the most buckets
    const int64_t e = uniform(p.block_expert[blockIdx.y]);
    p.b += e * b_rows * p.ldb;
    p.b_scales += e * (b_rows / kBlock) * p.sb_row;
    M = 0;  // a bucket's pairs come first
    while (M < kFewRows && (uint64_t)(int64_t)p.sorted[first + M] < (uint64_t)p.pairs) ++M;
  }

  // copies: rows 8 j + lane / 8 of the 16, whole lines, piece c of row x at c ^ ((x >> 1) & 7)
  const int piece = ((lane & 7) ^ (lane >> 4)) * 16;
  uint32_t woff[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int x = 8 * j + (lane >> 3);
    const int row = kPaired ? (j == 0 ? n0 + x : N + n0 + x - 8) : n0 + x;
    woff[j] = row < b_rows ? (uint32_t)(row * p.ldb) + (piece ^ (j * 64)) : kOut;
  }
  const __amdgpu_buffer_rsrc_t wres = __builtin_amdgcn_make_buffer_rsrc(
      (void*)p.b, 0, (int32_t)((b_rows - 1) * p.ldb + K), kBufferFlags);
  const __amdgpu_buffer_rsrc_t xres = __builtin_amdgcn_make_buffer_rsrc(
      (void*)p.a, 0, kFresh ? 0 : (int32_t)((M - 1) * p.lda + K), kBufferFlags);
  const uint32_t xoff = r < M ? (uint32_t)(r * p.lda) + 16 * q : kOut;

  u32x4 x[kFresh ? 1 : kD][2];
  // a stage's loads, all of them always issued, so that a wave's waits can count them
  constexpr int kLoads = kFresh ? 2 : 4;
  // this wave's stages, slice after slice; the next one to load
  const int per = wave < stages ? (stages - wave + kWaves - 1) / kWaves : 0, total = per * slices;
  int next_s = wave, next_slice = 0;
  auto load = [&](auto slot) {
    constexpr int d = decltype(slot)::value;
    const lds_bytes dst = ring[d] + wave * kSlot;
    const int s = next_s, slice = next_slice;
    const bool live = slice < slices && s < stages;
    const uint32_t from = (uint32_t)(slice * kStep * p.ldb) + (uint32_t)(s * kRow);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool in = live && (piece ^ (j * 64)) < K - s * kRow;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wres, (lds_ptr)(dst + j * 1024), 16,
                                               in ? woff[j] + from : kOut, 0, 0, 2);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (!kFresh) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = s * kRow + h * 64 + 16 * q < K;
        x[d][h] = __builtin_amdgcn_raw_buffer_load_b128(
            xres, in ? xoff + (uint32_t)(s * kRow + h * 64) : kOut, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    next_s += kWaves;
    if (next_s >= stages) next_s = wave, ++next_slice;
  };
  auto fill = [&] { each<kD>([&](auto d) { load(d); }); };

  const int stride = rows_code_stride(K), rows = kExperts ? kFewRows : M;
  float* const as = (float*)(qa + (kFresh ? rows * stride : 0));
  float* const bs = as + rows * stages;
  // scales into LDS; the first ones are asked for ahead of the ring's copies
  auto b_scale = [&](int i) {
    const int up = i >= stages;
    return p.b_scales[(int64_t)((up ? N + n0 : n0) / kBlock) * p.sb_row + i - up * stages];
  };
  const int b_count = (kPaired ? 2 : 1) * stages;
  const float b_first = (int)threadIdx.x < b_count ? b_scale(threadIdx.x) : 0.f;
  if constexpr (!kFresh) {
    constexpr int kPre = 8;
    float pre[kPre];
    const int count = M * stages;
#pragma unroll
    for (int i = 0; i < kPre; ++i) {
      const int at = i * kThreads + threadIdx.x;
      pre[i] = at < count ? p.a_scales[at % stages * p.a_rows + at / stages] : 0.f;
    }
    fill();
#pragma unroll
    for (int i = 0; i < kPre; ++i) {
      const int at = i * kThreads + threadIdx.x;
      if (at < count) as[at] = pre[i];
    }
    for (int at = kPre * kThreads + threadIdx.x; at < count; at += kThreads)
      as[at] = p.a_scales[at % stages * p.a_rows + at / stages];
  } else {
    // eights of a row over the threads, 16 a block; kAtOnce turns under way
    constexpr int kType = SRC == kBf16 ? MOE_TYPE_BF16 : MOE_TYPE_FP32, kAtOnce = 4;
    const int units = K / 8, turns = (stages * 16 + kThreads - 1) / kThreads;
    const int all = M * turns;
    for (int t = 0;; t += kAtOnce) {
      float v[kAtOnce][8];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int row = (t + i) / turns, u = (t + i) % turns * kThreads + threadIdx.x;
        if (t + i < all && u < units) {
          int64_t src = row;
          if constexpr (EPI == kSwiglu) src = p.sorted[first + row] / p.top_k;
          if constexpr (EPI == kPairs) src = first + row;
          load8<kType>(p.a, src * units + u, v[i]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i][k] = 0.f;
        }
      }
      if (t == 0) fill();
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int row = (t + i) / turns, u = (t + i) % turns * kThreads + threadIdx.x;
        const uint32_t field = scale_field(top_of_16(top8(v[i])));
        if (t + i < all && u < stages * 16) {
          *(u32x2*)(qa + row * stride + u * 8) = codes8(v[i], field);
          if ((u & 15) == 0) as[row * stages + u / 16] = scale_value(field);
        }
      }
      if (t + kAtOnce >= all) break;
    }
  }
  if ((int)threadIdx.x < b_count) bs[threadIdx.x] = b_first;
  for (int i = kThreads + threadIdx.x; i < b_count; i += kThreads) bs[i] = b_scale(i);
  wait_lgkm0();
  __builtin_amdgcn_s_barrier();  // (no wait for the ring's copies)
  __builtin_amdgcn_sched_barrier(0);

  f32x4 acc[1][1][1] = {{{f32x4{0.f, 0.f, 0.f, 0.f}}}};
  const int row = r < M ? r : 0;  // sums past the last row are not stored
  auto step = [&](auto slot, int s) {
    constexpr int d = decltype(slot)::value;
    const lds_bytes src = ring[d] + wave * kSlot;
    Frags<1> w, m;
    Wide<1> wide[1];
    ColumnScales<false, 1> cs[1];
    wait_vm<(kD - 1) * kLoads>();  // this stage's copies have landed
    __builtin_amdgcn_sched_barrier(0);
    w.read(src, 0, lane);
    cs[0].set(bs[kPaired && q >= 2 ? stages + s : s]);  // rows 4 q .. 4 q + 3: one square block
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (kFresh)
        m.v[0][h] = *(const u32x4*)(qa + row * stride + s * kRow + h * 64 + 16 * q);
      else
        m.v[0][h] = x[d][h];
    }
    const float sa[1] = {as[row * stages + s]};
    // the matrix units wait for memory anyway: the sums are fp32 for either result
    wide[0].set(w);
    mma_wide<false, 1, 1, 1>(acc, wide, m, sa, cs);
    hold(acc);
    wait_lgkm0();  // the place is read before the next copy into it goes out
    load(slot);
  };
  // lane (r, q) holds weight rows 4 q .. 4 q + 3 of A's row r
  float* const kept = (float*)(qa + rows_sums_at(kFresh, rows, K));  // fresh: [wave][slice][row][16]
  int s = wave, slice = 0;
  auto keep = [&] {
    if (r < M) *(f32x4*)&kept[((wave * slices + slice) * rows + r) * 16 + 4 * q] = acc[0][0][0];
    acc[0][0][0] = f32x4{0.f, 0.f, 0.f, 0.f};
    ++slice;
  };
  for (int n = 0; n < total; n += kD)
    each<kD>([&](auto d) {
      if (n + decltype(d)::value >= total) return;  // uniform: a wave's stages are its own
      step(d, s);
      s += kWaves;
      if (s < stages) return;
      s = wave;
      if constexpr (kFresh) keep();
    });
  if constexpr (kFresh)
    while (slice < slices) keep();  // a wave without stages: zeros

  wait_vm<0>();  // the copies past the last stage land before the LDS is given up or holds sums
  __syncthreads();
  const float* sums = kept;  // of wave 0; the others' `pitch` further each
  int pitch = slices * rows * 16;
  if constexpr (!kFresh) {
    *(f32x4*)&((float*)ring0)[wave * 256 + r * 16 + 4 * q] = acc[0][0][0];
    __syncthreads();
    sums = (const float*)ring0;
    pitch = 256;
  }
  const int count = (kFresh ? slices * M : M) * kStep;
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const int j = i % kStep, m = i / kStep % M, sl = i / (kStep * M);
    const int n = n0 + sl * kStep + j;
    if (n >= N) continue;
    const float* at = sums + (sl * rows + m) * 16 + j;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) v += at[k * pitch];
    if constexpr (kPaired) {
      float u = 0.f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) u += at[k * pitch + 8];
      ((float*)p.out)[(first + m) * N + n] = v * sigmoid(v) * u;
    } else if constexpr (EPI == kPairs) {
      ((float*)p.out)[(int64_t)p.sorted[first + m] * N + n] = v;
    } else if constexpr (EPI == kStoreF32) {
      ((float*)p.out)[(int64_t)m * N + n] = v;
    } else {
      ((uint16_t*)p.out)[(int64_t)m * N + n] = (uint16_t)pack2(v, 0.f);
    }
  }
#endif
}

template <Source SRC, Epilogue EPI>
hipError_t launch(const Product& p, int64_t buckets, hipStream_t stream) {
  constexpr bool kExperts = EPI == kSwiglu || EPI == kPairs;
  constexpr int kStep = rows_step(EPI), kD = kExperts ? kExpertsStages : kRowsStages;
  const int64_t rows = kExperts ? kFewRows : p.M, all = (p.N + kStep - 1) / kStep;
  const int slices = kExperts ? experts_slices(EPI, p.N, p.K, buckets) : 1;
  hipLaunchKernelGGL((rows_kernel<SRC, EPI, kD>),
                     dim3((unsigned)((all + slices - 1) / slices), (unsigned)buckets),
                     dim3(kThreads), rows_extra(SRC != kCodes, rows, p.K, slices), stream, p,
                     slices);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rows(Source source, Epilogue epilogue, const Product& p, hipStream_t stream) {
  if (source == kCodes)
    return epilogue == kStoreBf16 ? launch<kCodes, kStoreBf16>(p, 1, stream)
                                  : launch<kCodes, kStoreF32>(p, 1, stream);
  if (source == kBf16)
    return epilogue == kStoreBf16 ? launch<kBf16, kStoreBf16>(p, 1, stream)
                                  : launch<kBf16, kStoreF32>(p, 1, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_experts_rows(Epilogue epilogue, const Product& p, int64_t buckets,
                               hipStream_t stream) {
  if (epilogue == kSwiglu) return launch<kBf16, kSwiglu>(p, buckets, stream);
  if (epilogue == kPairs) return launch<kF32, kPairs>(p, buckets, stream);
  return hipErrorInvalidValue;
}

}  // namespace fp8
