// mxfp4.hip -- MXFP4 quantisation and its inverse (gfx950): blocks of 32 values
// along a row <-> one e8m0 scale byte and 32 e2m1 codes.
//
// Both are one pass over memory. A lane owns 8 consecutive values (16 bytes of
// bf16 or fp16, 32 of fp32; 4 bytes of codes), four neighbouring lanes a block.
// The largest magnitude is compared as bits (an unsigned maximum orders
// magnitudes, infinities and NaN on top), so e is its exponent field less 2,
// and v_cvt_scalef32_pk_fp4_f32 divides by 2^e, rounds to nearest even and
// saturates.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe_ffn.h"
#include "ffn_device.h"
#include "ffn_internal.h"

namespace ffn {
namespace {

constexpr int kThreads = 256;

template <int TYPE>
__device__ __forceinline__ void load8(const void* x, int64_t unit, float* v) {
  if constexpr (TYPE == MOE_TYPE_FP32) {
    const f32x4* p = (const f32x4*)x + 2 * unit;
    const f32x4 a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
    const u32x4 w = ((const u32x4*)x)[unit];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == MOE_TYPE_BF16) {
        v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
        v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
      } else {
        const h16x2 h = __builtin_bit_cast(h16x2, (uint32_t)w[i]);
        v[2 * i] = (float)h[0], v[2 * i + 1] = (float)h[1];
      }
    }
  }
}

// pad: 0, or the scale bytes of a row (width/32) where they go into padded rows
template <int TYPE>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const void* __restrict__ x,
                                                            int64_t units, int32_t pad,
                                                            uint32_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  // units is a multiple of 4: a block's lanes are all in or all out
  const int64_t u = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
  if (u >= units) return;
  float v[8];
  load8<TYPE>(x, u, v);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu;
    top = b > top ? b : top;
  }
  const uint32_t o1 = __shfl_xor(top, 1);
  top = o1 > top ? o1 : top;
  const uint32_t o2 = __shfl_xor(top, 2);
  top = o2 > top ? o2 : top;
  const uint32_t scale = mx_scale(top >> 23);
  const float unit = mx_unit(scale);
  uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], unit, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], unit, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], unit, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], unit, 3);
  if (scale == 255) c = 0;
  codes[u] = c;
  if ((u & 3) == 0) {
    const uint8_t byte = (uint8_t)scale;
    const int64_t b = u >> 2;
    if (pad == 0) {
      scales[b] = byte;
    } else {
      const int64_t row = b / pad;
      const int32_t at = (int32_t)(b - row * pad), stride = (pad + 7) / 8 * 8;
      scales[row * stride + at] = byte;
      if (at == pad - 1)
        for (int32_t i = pad; i < stride; ++i) scales[row * stride + i] = 127;
    }
  }
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint32_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales,
                                                              int64_t units,
                                                              void* __restrict__ out) {
  const int64_t u = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
  if (u >= units) return;
  const uint32_t c = codes[u];
  const int s = scales[u >> 2];
  float v[8];
  const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
  const f32x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
  const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
  const f32x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
  const float q[8] = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = s == 255 ? __builtin_nanf("") : ldexpf(q[i], s - 127);
  if constexpr (TYPE == MOE_TYPE_FP32) {
    f32x4* o = (f32x4*)out + 2 * u;
    o[0] = f32x4{v[0], v[1], v[2], v[3]};
    o[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 p = {v[2 * i], v[2 * i + 1]};
      if constexpr (TYPE == MOE_TYPE_BF16)
        w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
      else
        w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, h16x2));
    }
    ((u32x4*)out)[u] = w;
  }
}

// One thread a padded scale byte, of the first matrix and then of the second.
__global__ __launch_bounds__(kThreads) void pad_scales_kernel(
    const uint8_t* __restrict__ s0, int64_t n0, uint8_t* __restrict__ out0,
    const uint8_t* __restrict__ s1, int64_t n1, uint8_t* __restrict__ out1, int32_t blocks,
    int32_t stride) {
  int64_t u = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
  if (u >= n0 + n1) return;
  const bool second = u >= n0;
  if (second) u -= n0;
  const int64_t row = u / stride;
  const int32_t at = (int32_t)(u - row * stride);
  (second ? out1 : out0)[u] = at < blocks ? (second ? s1 : s0)[row * blocks + at] : 127;
}

// work-groups for `units` lanes: one dimension of a launch holds fewer than 2^32 lanes
dim3 grid_of(int64_t units) {
  const int64_t groups = (units + kThreads - 1) / kThreads;
  const int64_t y = (groups + (1 << 20) - 1) >> 20;
  return dim3((unsigned)((groups + y - 1) / y), (unsigned)y);
}

}  // namespace

hipError_t launch_mx_pad_scales(const uint8_t* s0, int64_t rows0, uint8_t* out0,
                                const uint8_t* s1, int64_t rows1, uint8_t* out1, int32_t width,
                                hipStream_t stream) {
  const int32_t stride = (int32_t)scale_stride(width);
  if (rows0 + rows1 == 0) return hipSuccess;
  hipLaunchKernelGGL(pad_scales_kernel, grid_of((rows0 + rows1) * stride), dim3(kThreads), 0,
                     stream, s0, rows0 * stride, out0, s1, rows1 * stride, out1, width / 32,
                     stride);
  return hipGetLastError();
}

hipError_t launch_mx_quantize(const void* x, int32_t type, int64_t rows, int32_t width,
                              uint8_t* codes, uint8_t* scales, bool padded, hipStream_t stream) {
  const int64_t units = rows * (width / 8);
  if (units == 0) return hipSuccess;
  const dim3 grid = grid_of(units), block(kThreads);
  const int32_t pad = padded && width % 256 ? width / 32 : 0;
  if (type == MOE_TYPE_BF16)
    hipLaunchKernelGGL(quantize_kernel<MOE_TYPE_BF16>, grid, block, 0, stream, x, units, pad,
                       (uint32_t*)codes, scales);
  else if (type == MOE_TYPE_FP16)
    hipLaunchKernelGGL(quantize_kernel<MOE_TYPE_FP16>, grid, block, 0, stream, x, units, pad,
                       (uint32_t*)codes, scales);
  else
    hipLaunchKernelGGL(quantize_kernel<MOE_TYPE_FP32>, grid, block, 0, stream, x, units, pad,
                       (uint32_t*)codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                int32_t width, int32_t type, void* out, hipStream_t stream) {
  const int64_t units = rows * (width / 8);
  if (units == 0) return hipSuccess;
  const dim3 grid = grid_of(units), block(kThreads);
  if (type == MOE_TYPE_BF16)
    hipLaunchKernelGGL(dequantize_kernel<MOE_TYPE_BF16>, grid, block, 0, stream,
                       (const uint32_t*)codes, scales, units, out);
  else if (type == MOE_TYPE_FP16)
    hipLaunchKernelGGL(dequantize_kernel<MOE_TYPE_FP16>, grid, block, 0, stream,
                       (const uint32_t*)codes, scales, units, out);
  else
    hipLaunchKernelGGL(dequantize_kernel<MOE_TYPE_FP32>, grid, block, 0, stream,
                       (const uint32_t*)codes, scales, units, out);
  return hipGetLastError();
}

}  // namespace ffn
