// ffn_small.hip -- the K-contiguous products for at most 64 rows (gfx950):
// decoding, where the time is the weights' way from memory.
//
// A work-group owns 16 weight rows (SwiGLU: 8 gate rows and their 8 up rows) and
// all rows of A: one, two or four 16 x 16 MFMA tiles. Its eight waves take the
// stages of K (128 bytes of a row) in turn, so that together they read whole
// kilobytes of each row; a wave keeps a ring of stages in flight in registers,
// loads straight into the MFMA's layout (lane (r = lane % 16, q = lane / 16):
// piece 4 step + q of row r) and never waits for another wave. At the end the
// waves' sums are added in LDS, in wave order.
//
// An A that is to be quantised (bf16, or the fp32 h of the block) is quantised
// by the work-group into LDS, four pieces a thread at a time; the ring's loads go
// out ahead of the last four's conversion, so a longer A is waited for first (8
// rows of 7168: three trips to memory before the first weights are asked for).
// Every work-group repeats it.
//
// bf16 is bound by memory and, below 100 MB, by how long a launch takes to fill
// and drain it: one token at 7168/2048 reads 59 MB in 12.6 us (4.7 TB/s) and 29
// MB in 8.8 us (3.3 TB/s). MXFP4 is bound by the way of A ahead of the weights: 8
// tokens at 7168/2048 16 MB in 11.1 us and 8 MB in 7.1 us, a wave waiting in 55%
// of its cycles. Past 16 rows it is bound by the loads' address path (64 cycles
// for 16 rows x 64 bytes; 32 x 4096 x 7168 in MXFP4 13.8 us, a wave waiting for
// its turn to issue in 62% of its cycles): 20 tokens at 1000/2000 13.3 us and 19.6
// with tiles, at 7168/2048 33.4 and 27.7; 64 tokens at 1000/2000 18.9 and 19.8.
// Its LDS conflicts (the sums' rows lie 64 bytes apart) are 200 to 450 cycles of a
// work-group's 8000 to 35000.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ffn_device.h"
#include "ffn_internal.h"

namespace ffn {
namespace {

constexpr int kWaves = 8, kThreads = kRowsThreads;
static_assert(kThreads == 64 * kWaves, "a work-group of the estimates");

#if defined(__HIP_DEVICE_COMPILE__)
template <int CTRL>
__device__ __forceinline__ uint32_t other_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
  return o > v ? o : v;
}
// One 16-byte piece of a block, the neighbouring four (bf16) or eight (fp32)
// lanes holding the whole: its codes (32 or 16 bits) and the block's scale.
template <bool F32>
__device__ __forceinline__ uint32_t quantize_piece(const u32x4& v, uint32_t* scale) {
  uint32_t top;
  if constexpr (F32) {
    top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t b = v[j] & 0x7fffffffu;
      top = b > top ? b : top;
    }
  } else {
    u16x2 m = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, (uint32_t)(v[j] & 0x7fff7fffu)));
    top = m[0] > m[1] ? m[0] : m[1];
  }
  top = other_max<0xB1>(top);                     // lane ^ 1
  top = other_max<0x4E>(top);                     // lane ^ 2
  if constexpr (F32) top = other_max<0x141>(top);  // the other four of eight
  *scale = mx_scale(top >> (F32 ? 23 : 7));
  const float unit = mx_unit(*scale);
  uint32_t c = 0;
  if constexpr (F32) {
    const f32x4 f = __builtin_bit_cast(f32x4, v);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[0], f[1], unit, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2], f[3], unit, 1);
  } else {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)v[0]), unit, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)v[1]), unit, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)v[2]), unit, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)v[3]), unit, 3);
  }
  return *scale == 255 ? 0 : c;
}
#endif

// A: as the product's operands (kAsIs), or bf16 / fp32 rows to quantise
enum AKind { kAsIs = 0, kFromBf16 = 1, kFromF32 = 2 };

// MT: 16-row tiles of A
template <AKind AK, bool MX, Epilogue EPI, int MT>
__global__ __launch_bounds__(kThreads, MT == 1 ? 4 : 2) void rows_kernel(const Product p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr bool kPaired = EPI == kSwiglu || EPI == kSwigluF32;
  // stages in flight per wave, by what their registers leave
  constexpr int kD = AK == kFromF32 ? 3 : MT == 1 ? 5 : MT == 2 ? 4 : 3;
  // quantised A (codes, then bytes), and in its place at the end the waves' sums
  extern __shared__ __attribute__((aligned(16))) uint8_t qa[];
  float* const sums = (float*)qa;

  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int M = (int)p.M, N = p.N, kb = (int)(MX ? p.K / 2 : 2 * p.K);  // bytes of a row
  const int n0 = blockIdx.x * (kPaired ? 8 : 16);
  const int blocks = (int)(p.K / 32), stages = (kb + 127) / 128;

  const int row = kPaired ? (r < 8 ? n0 + r : N + n0 + r - 8) : n0 + r;
  const int rows = kPaired ? 2 * N : N;
  const uint32_t woff = row < rows ? (uint32_t)row * kb + 16 * q : kOut;
  const uint32_t wsoff = row < rows ? (uint32_t)row * blocks + q : kOut;
  uint32_t xoff[MT], xsoff[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    xoff[i] = 16 * i + r < M ? (uint32_t)(16 * i + r) * kb + 16 * q : kOut;
    xsoff[i] = 16 * i + r < M ? (uint32_t)(16 * i + r) * blocks + q : kOut;
  }
  const __amdgpu_buffer_rsrc_t wres =
      __builtin_amdgcn_make_buffer_rsrc((void*)p.b, 0, rows * kb, kBufferFlags);
  const __amdgpu_buffer_rsrc_t wsres =
      __builtin_amdgcn_make_buffer_rsrc((void*)p.b_scales, 0, MX ? rows * blocks : 0, kBufferFlags);
  const __amdgpu_buffer_rsrc_t xres =
      __builtin_amdgcn_make_buffer_rsrc((void*)p.a, 0, M * kb, kBufferFlags);
  const __amdgpu_buffer_rsrc_t xsres = __builtin_amdgcn_make_buffer_rsrc(
      (void*)p.a_scales, 0, MX && AK == kAsIs ? M * blocks : 0, kBufferFlags);

  u32x4 w[kD][2], x[kD][2][MT];
  uint32_t ws[kD][2], xs[kD][2][MT];
  auto load = [&](int d, int s) {
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const int at = s * 128 + st * 64;
      const bool in = at + 16 * q < kb;
      if constexpr (AK == kAsIs)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          x[d][st][i] = __builtin_amdgcn_raw_buffer_load_b128(xres, in ? xoff[i] + at : kOut, 0, 0);
      w[d][st] = __builtin_amdgcn_raw_buffer_load_b128(wres, in ? woff + at : kOut, 0, 0);
      if constexpr (MX) {
        const int b = 8 * s + 4 * st;
        if constexpr (AK == kAsIs)
#pragma unroll
          for (int i = 0; i < MT; ++i)
            xs[d][st][i] = __builtin_amdgcn_raw_buffer_load_b8(xsres, in ? xsoff[i] + b : kOut, 0, 0);
        ws[d][st] = __builtin_amdgcn_raw_buffer_load_b8(wsres, in ? wsoff + b : kOut, 0, 0);
      }
    }
  };
  auto fill = [&] {
#pragma unroll
    for (int d = 0; d < kD; ++d) load(d, wave + d * kWaves);
  };

  const int cstride = rows_code_stride(p.K), bstride = rows_byte_stride(p.K);
  uint8_t* qbytes = qa + M * cstride;
  if constexpr (AK == kAsIs) {
    fill();
  } else {
    // The rows' 16-byte pieces over the threads: 2^sh threads a row (all of them
    // where it has more pieces), kAtOnce loads each under way, the last ones
    // ahead of the ring's. Pieces past K, to a whole stage, are zeros with a
    // finite scale.
    constexpr int kSize = AK == kFromF32 ? 4 : 2;       // bytes of a value
    constexpr int kLanes = 2 * kSize;                   // lanes of a block
    constexpr int kAtOnce = 4;
    const int have = blocks * kLanes, pieces = (blocks + 7) / 8 * 8 * kLanes;
    const int sh = pieces >= kThreads ? 9 : 32 - __builtin_clz(pieces - 1);
    const int across = 1 << sh, down = kThreads >> sh;  // threads a row, rows at once
    const int t0 = threadIdx.x >> sh, c0 = threadIdx.x & (across - 1);
    const int turns = (pieces + across - 1) >> sh;      // a row's
    const int total = (M + down - 1) / down * turns;
    const __amdgpu_buffer_rsrc_t ares = __builtin_amdgcn_make_buffer_rsrc(
        (void*)p.a, 0, M * have * 16, kBufferFlags);
    int t = t0, c = c0, turn = 0;
    auto next = [&](int& t, int& c, int& turn) {
      c += across;
      if (++turn == turns) turn = 0, c = c0, t += down;
    };
    for (int first = 0;; first += kAtOnce) {
      u32x4 v[kAtOnce];
      int tl = t, cl = c, turnl = turn;
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const bool in = first + j < total && tl < M && cl < have;
        v[j] = __builtin_amdgcn_raw_buffer_load_b128(ares, in ? (tl * have + cl) * 16 : kOut, 0, 0);
        next(tl, cl, turnl);
      }
      const bool last = first + kAtOnce >= total;
      if (last) fill();
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        uint32_t scale;
        const uint32_t code = quantize_piece<AK == kFromF32>(v[j], &scale);
        if (first + j < total && t < M && c < pieces) {
          if constexpr (AK == kFromF32)
            *(uint16_t*)(qa + t * cstride + 2 * c) = (uint16_t)code;
          else
            *(uint32_t*)(qa + t * cstride + 4 * c) = code;
          if (c % kLanes == 0) qbytes[t * bstride + c / kLanes] = (uint8_t)scale;
        }
        next(t, c, turn);
      }
      if (last) break;
    }
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
  }

  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s = wave; s < stages; s += kD * kWaves) {
#pragma unroll
    for (int d = 0; d < kD; ++d) {
      const int at = s + d * kWaves;
      if (at >= stages) break;  // uniform: a wave's stages are its own
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          if constexpr (MX) {
            u32x4 xv;
            uint32_t xb;
            if constexpr (AK == kAsIs) {
              xv = x[d][st][i], xb = xs[d][st][i];
            } else {
              // rows past the last: any, their sums are not stored
              const int row = 16 * i + r < M ? 16 * i + r : M - 1;
              xv = *(const u32x4*)(qa + row * cstride + at * 128 + st * 64 + 16 * q);
              xb = qbytes[row * bstride + 8 * at + 4 * st + q];
            }
            acc[i] = mfma_mx<0, 0>(w[d][st], xv, acc[i], ws[d][st], xb);
          } else {
            acc[i] = mfma(w[d][st], x[d][st][i], acc[i]);
          }
        }
      load(d, at + kD * kWaves);
    }
  }

  // lane (r, q) holds weight rows 4 q .. 4 q + 3 of A's row 16 i + r
  if constexpr (AK != kAsIs) __syncthreads();  // A is read to the end
#pragma unroll
  for (int i = 0; i < MT; ++i)
    *(f32x4*)&sums[(wave * MT + i) * 256 + r * 16 + 4 * q] = acc[i];
  __syncthreads();
  if constexpr (kPaired) {
    for (int i = threadIdx.x; i < 128 * MT; i += kThreads) {
      const int m = i >> 3, j = i & 7;
      if (m >= M) break;
      float g = 0.f, u = 0.f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        g += sums[k * MT * 256 + m * 16 + j];
        u += sums[k * MT * 256 + m * 16 + 8 + j];
      }
      const float h = g * sigmoid(g) * u;
      const int64_t at = (int64_t)m * N + n0 + j;
      if constexpr (EPI == kSwigluF32) {
        ((float*)p.out)[at] = h;
      } else {
        ((uint16_t*)p.out)[at] = (uint16_t)pack2(h, 0.f);  // as the matrix units take it
        if (p.aux) {
          float* gu = (float*)p.aux + (int64_t)m * 2 * N + n0 + j;
          gu[0] = g;
          gu[N] = u;
        }
      }
    }
  } else {
    for (int i = threadIdx.x; i < 256 * MT; i += kThreads) {
      const int m = i >> 4, n = n0 + (i & 15);
      if (m >= M) break;
      if (n >= N) continue;
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) v += sums[k * MT * 256 + i];
      if constexpr (EPI == kStoreF32)
        ((float*)p.out)[(int64_t)m * N + n] = v;
      else
        ((uint16_t*)p.out)[(int64_t)m * N + n] = (uint16_t)pack2(v, 0.f);
    }
  }
#endif
}

template <AKind AK, bool MX, Epilogue EPI, int MT>
hipError_t launch_tiles(const Product& p, hipStream_t stream) {
  const unsigned groups = EPI == kSwiglu || EPI == kSwigluF32 ? (p.N + 7) / 8 : (p.N + 15) / 16;
  const size_t a = AK == kAsIs ? 0 : p.M * (rows_code_stride(p.K) + rows_byte_stride(p.K));
  const size_t lds = std::max<size_t>(a, kWaves * MT * 256 * sizeof(float));
  hipLaunchKernelGGL((rows_kernel<AK, MX, EPI, MT>), dim3(groups), dim3(kThreads), lds, stream,
                     p);
  return hipGetLastError();
}
template <AKind AK, bool MX, Epilogue EPI>
hipError_t launch(const Product& p, hipStream_t stream) {
  if (p.M <= 16) return launch_tiles<AK, MX, EPI, 1>(p, stream);
  if (AK == kFromBf16) return hipErrorInvalidValue;  // rows_fit takes 16 rows of those at most
  if constexpr (AK != kFromBf16) {
    if (p.M <= 32) return launch_tiles<AK, MX, EPI, 2>(p, stream);
    if (p.M <= 64) return launch_tiles<AK, MX, EPI, 4>(p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_rows(Epilogue epilogue, const Product& p, hipStream_t stream) {
  if (epilogue == kSwiglu) return launch<kAsIs, false, kSwiglu>(p, stream);
  if (epilogue == kStoreBf16) return launch<kAsIs, false, kStoreBf16>(p, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_rows_mx(Epilogue epilogue, AType a, const Product& p, hipStream_t stream) {
  if (epilogue == kSwigluF32 && a == kABf16) return launch<kFromBf16, true, kSwigluF32>(p, stream);
  if (epilogue == kSwigluF32 && a == kAAsIs) return launch<kAsIs, true, kSwigluF32>(p, stream);
  if (epilogue == kStoreBf16 && a == kAF32) return launch<kFromF32, true, kStoreBf16>(p, stream);
  if (epilogue == kStoreBf16 && a == kABf16) return launch<kFromBf16, true, kStoreBf16>(p, stream);
  if (epilogue == kStoreF32 && a == kABf16) return launch<kFromBf16, true, kStoreF32>(p, stream);
  if (epilogue == kStoreBf16) return launch<kAsIs, true, kStoreBf16>(p, stream);
  if (epilogue == kStoreF32) return launch<kAsIs, true, kStoreF32>(p, stream);
  return hipErrorInvalidValue;
}

}  // namespace ffn
