// mxfp4.hip -- MXFP4 quantisation and its inverse (gfx950): blocks of 32 values
// along a row <-> one e8m0 scale byte and 32 e2m1 codes.
//
// Both are one pass over memory. A lane owns 8 consecutive values (16 bytes of
// bf16 or fp16, 32 of fp32; 4 bytes of codes), four neighbouring lanes a block.
// The largest magnitude is compared as bits (an unsigned maximum orders
// magnitudes, infinities and NaN on top), so e is its exponent field less 2,
// and v_cvt_scalef32_pk_fp4_f32 divides by 2^e, rounds to nearest even and
// saturates. Bound by memory: 4096 x 7168 of fp32 (133 MB) 22.5 us to codes and
// 22.9 us back, 5.9 and 5.8 TB/s; 8 x 7168 of bf16 2.4 us, a launch.
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

// Eight values of a block -> their codes; *byte: the block's scale
template <int TYPE>
__device__ __forceinline__ uint32_t quantize8(const void* x, int64_t u, uint32_t* byte) {
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
  *byte = mx_scale(top >> 23);
  const float unit = mx_unit(*byte);
  uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], unit, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], unit, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], unit, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], unit, 3);
  return *byte == 255 ? 0 : c;
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const void* __restrict__ x,
                                                            int64_t units,
                                                            uint32_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  // units is a multiple of 4: a block's lanes are all in or all out
  const int64_t u = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
  if (u >= units) return;
  uint32_t byte;
  codes[u] = quantize8<TYPE>(x, u, &byte);
  if ((u & 3) == 0) scales[u >> 2] = (uint8_t)byte;
}

// The first work-groups copy scales into the order by stage, one wave 64 rows
// of four stages (the rows' bytes come in runs of 32 and leave 512 at a time);
// they wait on memory, so they start ahead of those that quantise x. 4096 x 7168
// of bf16 with a matrix's scales (77 MB) 16.2 us, 4.8 TB/s. Rows of K/32 bytes
// that start anywhere are gathered byte by byte: 55 KB (777 and 1000 rows of 992)
// take 5.4 us, a wave waiting in 82% of its cycles.
struct Prepare {
  const void* x;
  int64_t units, rows;
  int32_t blocks;  // of a row of x
  uint32_t* codes;
  uint8_t* scales;
  int64_t groups0, groups;  // work-groups of s0, of s0 and s1
  ScaleCopy s0, s1;
};
__global__ __launch_bounds__(kThreads) void prepare_kernel(const Prepare p) {
  const int64_t group = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (group >= p.groups) {
    const int64_t u = (group - p.groups) * kThreads + threadIdx.x;
    if (u >= p.units) return;
    uint32_t byte;
    p.codes[u] = quantize8<MOE_TYPE_BF16>(p.x, u, &byte);
    if ((u & 3) != 0) return;
    const int64_t b = u >> 2, row = b / p.blocks;
    const int32_t at = (int32_t)(b - row * p.blocks);
    uint8_t* dst = p.scales + ((at >> 3) * scale_rows(p.rows) + row) * 8;
    dst[at & 7] = (uint8_t)byte;
    if (at == p.blocks - 1)
      for (int i = (at & 7) + 1; i < 8; ++i) dst[i] = 127;
    return;
  }
  const bool second = group >= p.groups0;
  const ScaleCopy& s = second ? p.s1 : p.s0;
  const int64_t wave = (group - (second ? p.groups0 : 0)) * (kThreads / 64) + (threadIdx.x >> 6);
  const int64_t stages = scale_stages(s.width), quads = (stages + 3) / 4;
  const int64_t row = wave / quads * 64 + (threadIdx.x & 63), s0 = wave % quads * 4;
  if (row >= s.rows) return;
  const int32_t blocks = s.width / 32;
  const uint8_t* src = s.src + row * blocks;
  const int64_t pitch = scale_rows(s.rows) * 8;
  uint8_t* dst = s.dst + row * 8 + s0 * pitch;
  const int count = (int)(stages - s0 < 4 ? stages - s0 : 4);
  u32x2 v[4];
  if (blocks % 8 == 0 && ((uintptr_t)s.src & 7) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < count) v[i] = *(const u32x2*)(src + (s0 + i) * 8);
  } else {  // rows start at any byte, and the last stage may be short
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = u32x2{0x7f7f7f7fu, 0x7f7f7f7fu};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t b = (s0 + i) * 8 + j;
        const uint32_t byte = b < blocks ? src[b] : 127u;
        v[i][j / 4] = (v[i][j / 4] & ~(0xffu << (8 * (j & 3)))) | (byte << (8 * (j & 3)));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < count) *(u32x2*)(dst + i * pitch) = v[i];
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

// a launch of `groups` work-groups: one dimension holds fewer than 2^32 lanes
dim3 grid_of(int64_t groups) {
  const int64_t y = (groups + (1 << 20) - 1) >> 20;
  return dim3((unsigned)((groups + y - 1) / y), (unsigned)y);
}

}  // namespace

hipError_t launch_mx_prepare(const void* x, int64_t rows, int32_t width, uint8_t* codes,
                             uint8_t* scales, const ScaleCopy& s0, const ScaleCopy& s1,
                             hipStream_t stream) {
  auto copy_groups = [](const ScaleCopy& s) {
    const int64_t waves = (s.rows + 63) / 64 * ((scale_stages(s.width) + 3) / 4);
    return s.src ? (waves + kThreads / 64 - 1) / (kThreads / 64) : (int64_t)0;
  };
  Prepare p{};
  p.x = x;
  p.units = x ? rows * (width / 8) : 0;
  p.rows = rows;
  p.blocks = width / 32;
  p.codes = (uint32_t*)codes;
  p.scales = scales;
  p.groups0 = copy_groups(s0);
  p.groups = p.groups0 + copy_groups(s1);
  p.s0 = s0;
  p.s1 = s1;
  const int64_t total = p.groups + (p.units + kThreads - 1) / kThreads;
  if (total == 0) return hipSuccess;
  hipLaunchKernelGGL(prepare_kernel, grid_of(total), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_mx_quantize(const void* x, int32_t type, int64_t rows, int32_t width,
                              uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  const int64_t units = rows * (width / 8);
  if (units == 0) return hipSuccess;
  const dim3 grid = grid_of((units + kThreads - 1) / kThreads), block(kThreads);
  if (type == MOE_TYPE_BF16)
    hipLaunchKernelGGL(quantize_kernel<MOE_TYPE_BF16>, grid, block, 0, stream, x, units,
                       (uint32_t*)codes, scales);
  else if (type == MOE_TYPE_FP16)
    hipLaunchKernelGGL(quantize_kernel<MOE_TYPE_FP16>, grid, block, 0, stream, x, units,
                       (uint32_t*)codes, scales);
  else
    hipLaunchKernelGGL(quantize_kernel<MOE_TYPE_FP32>, grid, block, 0, stream, x, units,
                       (uint32_t*)codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                int32_t width, int32_t type, void* out, hipStream_t stream) {
  const int64_t units = rows * (width / 8);
  if (units == 0) return hipSuccess;
  const dim3 grid = grid_of((units + kThreads - 1) / kThreads), block(kThreads);
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
