// fp8.hip -- FP8 block quantisation, its inverse, and the transposes that the
// gradients read (gfx950).
//
// One pass over memory each. The largest magnitude is compared as bits (an
// unsigned maximum orders magnitudes, infinities and NaN on top); the scale is a
// power of two, so that dividing by it is exact and v_cvt_pk_fp8_f32 rounds once.
// Bound by memory: 4096 x 7168 of fp32 (147 MB) 25.5 us to codes in 128 x 128 blocks
// and 26.1 us back, 5.8 and 5.6 TB/s; of bf16 to codes in 1 x 128 blocks (88 MB) 19 us,
// 4.6 TB/s, a wave waiting in 75% of its cycles; 8 x 7168 of bf16 2.5 us, a launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/moe_fp8.h"
#include "fp8_device.h"
#include "fp8_internal.h"

namespace fp8 {
namespace {

constexpr int kThreads = 256;

template <int TYPE>
__device__ __forceinline__ void store8(void* x, int64_t unit, const float* v) {
  if constexpr (TYPE == MOE_TYPE_FP32) {
    f32x4* o = (f32x4*)x + 2 * unit;
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
    ((u32x4*)x)[unit] = w;
  }
}

// 1 x 128 blocks: 16 lanes a block, a work-group 16 rows of NB blocks, so that the
// scales of a stage leave 16 at a time.
template <int TYPE, int NB>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const void* __restrict__ x,
                                                                 int64_t rows, int32_t width,
                                                                 uint8_t* __restrict__ codes,
                                                                 float* __restrict__ scales) {
  const int32_t blocks = (width + kBlock - 1) / kBlock, units = width / 8;
  const int64_t row = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * 16 + (threadIdx.x >> 4);
  const int b0 = blockIdx.x * NB, at = threadIdx.x & 15;
  if (row >= rows) return;  // all 16 lanes of a row
  float v[NB][8];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int u = (b0 + i) * 16 + at;
    if (u < units) {
      load8<TYPE>(x, row * units + u, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int u = (b0 + i) * 16 + at;
    const uint32_t field = scale_field(top_of_16(top8(v[i])));
    if (u < units) ((u32x2*)codes)[row * units + u] = codes8(v[i], field);
    if (at == 0 && b0 + i < blocks) scales[(int64_t)(b0 + i) * rows + row] = scale_value(field);
  }
}

// 128 x 128 blocks: a work-group a block, its values in registers
template <int TYPE>
__global__ __launch_bounds__(kThreads) void quantize_square_kernel(const void* __restrict__ x,
                                                                   int64_t rows, int32_t width,
                                                                   uint8_t* __restrict__ codes,
                                                                   float* __restrict__ scales) {
  __shared__ uint32_t tops[kThreads / 64];
  const int32_t units = width / 8, u = blockIdx.x * 16 + (threadIdx.x & 15);
  const int64_t block_row = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
  if (block_row * kBlock >= rows) return;
  const int64_t row0 = block_row * kBlock + (threadIdx.x >> 4);
  float v[8][8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (u < units && row0 + 16 * i < rows) {
      load8<TYPE>(x, (row0 + 16 * i) * units + u, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) top = larger(top, top8(v[i]));
  top = top_of_16(top);
  top = larger(top, __shfl_xor(top, 16));
  top = larger(top, __shfl_xor(top, 32));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  top = larger(larger(tops[0], tops[1]), larger(tops[2], tops[3]));
  const uint32_t field = scale_field(top);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (u < units && row0 + 16 * i < rows)
      ((u32x2*)codes)[(row0 + 16 * i) * units + u] = codes8(v[i], field);
  if (threadIdx.x == 0) scales[block_row * gridDim.x + blockIdx.x] = scale_value(field);
}

// 16 rows of NB blocks a work-group, as the codes were made
template <int TYPE, int NB, bool SQUARE>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t* __restrict__ codes,
                                                              const float* __restrict__ scales,
                                                              int64_t rows, int32_t width,
                                                              void* __restrict__ out) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int32_t blocks = (width + kBlock - 1) / kBlock, units = width / 8;
  const int64_t row = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * 16 + (threadIdx.x >> 4);
  const int b0 = blockIdx.x * NB, at = threadIdx.x & 15;
  if (row >= rows) return;
  u32x2 c[NB];
  float s[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int u = (b0 + i) * 16 + at;
    if (u >= units) continue;
    c[i] = ((const u32x2*)codes)[row * units + u];
    s[i] = scales[SQUARE ? row / kBlock * blocks + b0 + i : (int64_t)(b0 + i) * rows + row];
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int u = (b0 + i) * 16 + at;
    if (u >= units) continue;
    float v[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i][j], false);
      const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i][j], true);
      v[4 * j] = lo[0] * s[i], v[4 * j + 1] = lo[1] * s[i];
      v[4 * j + 2] = hi[0] * s[i], v[4 * j + 3] = hi[1] * s[i];
    }
    store8<TYPE>(out, row * units + u, v);
  }
#endif
}

// A tile of 128 rows on its way to being 128 bytes of a column: 32 words of four
// rows, columns 33 words apart. The eight columns that a wave writes are 16 apart, 528
// words, 16 banks of 64: the eight words of columns 64 apart meet, two ways; so do some of the
// eight neighbouring columns that it reads. Conflicts are 56% of the LDS's busy cycles in
// prepare_kernel, where the LDS is busy in 14 to 39%, and memory is what bounds it.
[[maybe_unused]] constexpr int kPitch = 33;

#if defined(__HIP_DEVICE_COMPILE__)
__device__ __forceinline__ void store_columns(const uint32_t* words, int64_t rows, int32_t width,
                                              int64_t block, int64_t col0, uint8_t* codes) {
  const int64_t pitch = blocks_of(rows) * kBlock;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = i * 32 + (threadIdx.x >> 3), w = (threadIdx.x & 7) * 4;
    const uint32_t* p = words + c * kPitch + w;
    const u32x4 v = {p[0], p[1], p[2], p[3]};
    if (col0 + c < width) *(u32x4*)(codes + (col0 + c) * pitch + block * kBlock + 4 * w) = v;
  }
}

// A block of 128 rows x 128 columns of x bf16, a thread four rows of 16 columns: quantised along
// the columns into the transpose (see launch_prepare), and where row_codes is given along the
// rows too, in rows of 128 blocks_of(width) bytes
__device__ __forceinline__ void quantize_block(uint32_t* words, uint32_t (*tops)[128],
                                               const void* x, int64_t rows, int32_t width,
                                               int64_t block, int64_t column_block,
                                               uint8_t* row_codes, float* row_scales,
                                               uint8_t* codes, float* scales) {
  const int32_t units = width / 8, across = (width + kBlock - 1) / kBlock;
  const int g = threadIdx.x >> 3, c16 = threadIdx.x & 7;
  const int64_t u = column_block * 16 + 2 * c16, row0 = block * kBlock + 4 * g;
  float v[4][16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (u + h < units && row0 + i < rows) {
        load8<MOE_TYPE_BF16>(x, (row0 + i) * units + u + h, v[i] + 8 * h);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][8 * h + j] = 0.f;
      }
    }
  if (row_codes) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t top = larger(top8(v[i]), top8(v[i] + 8));
      top = with_lane<0xB1>(top);   // lane ^ 1
      top = with_lane<0x4E>(top);   // lane ^ 2
      top = with_lane<0x141>(top);  // mirrored in eights
      const uint32_t field = scale_field(top);
      const u32x2 lo = codes8(v[i], field), hi = codes8(v[i] + 8, field);
      const int64_t row = row0 + i;
      if (row < rows) {
        *(u32x4*)(row_codes + (row * across + column_block) * kBlock + 16 * c16) =
            u32x4{lo[0], lo[1], hi[0], hi[1]};
        if (c16 == 0) row_scales[column_block * rows + row] = scale_value(field);
      }
    }
  }
  if (!codes) return;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    uint32_t top = larger(larger(magnitude(v[0][j]), magnitude(v[1][j])),
                          larger(magnitude(v[2][j]), magnitude(v[3][j])));
    top = larger(top, __shfl_xor(top, 8));
    top = larger(top, __shfl_xor(top, 16));
    top = larger(top, __shfl_xor(top, 32));
    if ((threadIdx.x & 63) < 8) tops[threadIdx.x >> 6][c16 * 16 + j] = top;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int c = c16 * 16 + j;
    const uint32_t field =
        scale_field(larger(larger(tops[0][c], tops[1][c]), larger(tops[2][c], tops[3][c])));
    const float col[4] = {v[0][j], v[1][j], v[2][j], v[3][j]};
    words[c * kPitch + g] = field == 255 ? 0 : pack4(col, scale_inverse(field));
    if (g == 0 && column_block * kBlock + c < width)
      scales[block * width + column_block * kBlock + c] = scale_value(field);
  }
  __syncthreads();
  store_columns(words, rows, width, block, column_block * kBlock, codes);
}

// 128 rows x 128 columns of codes, transposed: a thread four rows of 16 columns
__device__ __forceinline__ void transpose_block(uint32_t* words, const uint8_t* codes,
                                                int64_t rows, int32_t width, int64_t block,
                                                int64_t column_block, uint8_t* out) {
  const int32_t units = width / 16;
  const int g = threadIdx.x >> 3, c16 = threadIdx.x & 7;
  const int64_t u = column_block * 8 + c16, row0 = block * kBlock + 4 * g;
  u32x4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = u < units && row0 + i < rows ? ((const u32x4*)codes)[(row0 + i) * units + u]
                                        : u32x4{0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // bytes (row i, column 4 j + b) -> word of column 4 j + b
    const uint32_t lo01 = __builtin_amdgcn_perm(v[1][j], v[0][j], 0x05010400u);
    const uint32_t hi01 = __builtin_amdgcn_perm(v[1][j], v[0][j], 0x07030602u);
    const uint32_t lo23 = __builtin_amdgcn_perm(v[3][j], v[2][j], 0x05010400u);
    const uint32_t hi23 = __builtin_amdgcn_perm(v[3][j], v[2][j], 0x07030602u);
    uint32_t* w = words + (c16 * 16 + 4 * j) * kPitch + g;
    w[0] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
    w[kPitch] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
    w[2 * kPitch] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
    w[3 * kPitch] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
  }
  __syncthreads();
  store_columns(words, rows, width, block, column_block * kBlock, out);
}
#endif

// All that the gradients' products read, in one launch: blocks of 128 x 128 of B's codes, of
// dout and of a. 4096 x 4096 x 7168 (222 MB) 58 us, 3.8 TB/s, a wave waiting for memory in 74% of
// its cycles (four launches took 71 us); 201 x 1360 x 1008 11 us, which is one trip to memory, the
// columns' maxima over the waves, and the way back (four launches 19 us).
__global__ __launch_bounds__(kThreads) void prepare_kernel(const Prepare p, const int64_t first_dout,
                                                           const int64_t first_a,
                                                           const int64_t end) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ uint32_t words[128 * kPitch];
  __shared__ uint32_t tops[kThreads / 64][128];
  const int64_t group = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (group >= end) return;
  const int64_t wide = blocks_of(p.width), high = blocks_of(p.cols);
  if (group < first_dout) {
    transpose_block(words, p.b, p.cols, p.width, group / wide, group % wide, p.b_t);
  } else if (group < first_a) {
    const int64_t i = group - first_dout;
    quantize_block(words, tops, p.dout, p.rows, p.cols, i / high, i % high, p.dout_codes,
                   p.dout_scales, p.dout_t, p.dout_t_scales);
  } else {
    const int64_t i = group - first_a;
    quantize_block(words, tops, p.a, p.rows, p.width, i / wide, i % wide, nullptr, nullptr, p.a_t,
                   p.a_t_scales);
  }
#endif
}

// `down` work-groups of rows over y and z (65535 a dimension at most); across fits x
dim3 grid_of(int64_t across, int64_t down) {
  const int64_t z = (down + 65534) / 65535;
  return dim3((unsigned)across, (unsigned)((down + z - 1) / z), (unsigned)z);
}

template <typename F>
hipError_t with_type(int32_t type, F&& f) {
  if (type == MOE_TYPE_BF16)
    f(std::integral_constant<int, MOE_TYPE_BF16>{});
  else if (type == MOE_TYPE_FP16)
    f(std::integral_constant<int, MOE_TYPE_FP16>{});
  else
    f(std::integral_constant<int, MOE_TYPE_FP32>{});
  return hipGetLastError();
}
__global__ __launch_bounds__(kThreads) void clear_kernel(u32x4* __restrict__ out, int64_t units) {
  const int64_t u = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
  if (u < units) out[u] = u32x4{0, 0, 0, 0};
}

// Blocks of a row that a work-group takes: four, with their loads in flight together, once
// that still leaves work-groups for every CU
bool four_blocks(int64_t rows, int32_t width) {
  return (rows + 15) / 16 * ((blocks_of(width) + 3) / 4) >= 512;
}
template <int TYPE>
void quantize_rows(const void* x, int64_t rows, int32_t width, uint8_t* codes,
                   float* scales, hipStream_t stream) {
  const int64_t blocks = blocks_of(width), down = (rows + 15) / 16;
  if (four_blocks(rows, width))
    hipLaunchKernelGGL((quantize_rows_kernel<TYPE, 4>), grid_of((blocks + 3) / 4, down),
                       dim3(kThreads), 0, stream, x, rows, width, codes, scales);
  else
    hipLaunchKernelGGL((quantize_rows_kernel<TYPE, 1>), grid_of(blocks, down), dim3(kThreads), 0,
                       stream, x, rows, width, codes, scales);
}

}  // namespace

hipError_t launch_quantize(const void* x, int32_t type, int64_t rows, int32_t width, int32_t block,
                           uint8_t* codes, float* scales, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  return with_type(type, [&](auto t) {
    constexpr int TYPE = decltype(t)::value;
    if (block != 1)
      hipLaunchKernelGGL((quantize_square_kernel<TYPE>), grid_of(blocks_of(width), blocks_of(rows)),
                         dim3(kThreads), 0, stream, x, rows, width, codes, scales);
    else
      quantize_rows<TYPE>(x, rows, width, codes, scales, stream);
  });
}

hipError_t launch_clear(void* out, int64_t bytes, hipStream_t stream) {
  const int64_t units = bytes / 16, groups = (units + kThreads - 1) / kThreads;
  if (groups == 0) return hipSuccess;
  hipLaunchKernelGGL(clear_kernel, grid_of((groups + 65534) / 65535, groups < 65535 ? groups : 65535),
                     dim3(kThreads), 0, stream, (u32x4*)out, units);
  return hipGetLastError();
}

hipError_t launch_dequantize(const uint8_t* codes, const float* scales, int64_t rows,
                             int32_t width, int32_t block, int32_t type, void* out,
                             hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const bool four = four_blocks(rows, width);
  const dim3 grid = grid_of(four ? (blocks_of(width) + 3) / 4 : blocks_of(width), (rows + 15) / 16);
  return with_type(type, [&](auto t) {
    constexpr int TYPE = decltype(t)::value;
    if (block != 1 && four)
      hipLaunchKernelGGL((dequantize_kernel<TYPE, 4, true>), grid, dim3(kThreads), 0, stream,
                         codes, scales, rows, width, out);
    else if (block != 1)
      hipLaunchKernelGGL((dequantize_kernel<TYPE, 1, true>), grid, dim3(kThreads), 0, stream,
                         codes, scales, rows, width, out);
    else if (four)
      hipLaunchKernelGGL((dequantize_kernel<TYPE, 4, false>), grid, dim3(kThreads), 0, stream,
                         codes, scales, rows, width, out);
    else
      hipLaunchKernelGGL((dequantize_kernel<TYPE, 1, false>), grid, dim3(kThreads), 0, stream,
                         codes, scales, rows, width, out);
  });
}

hipError_t launch_prepare(const Prepare& p, hipStream_t stream) {
  const int64_t down = blocks_of(p.rows);
  const int64_t first_dout = p.b_t ? blocks_of(p.cols) * blocks_of(p.width) : 0;
  const int64_t first_a = first_dout + down * blocks_of(p.cols);
  const int64_t end = first_a + (p.a_t ? down * blocks_of(p.width) : 0);
  const int64_t y = (end + (1 << 20) - 1) >> 20;
  hipLaunchKernelGGL(prepare_kernel, dim3((unsigned)((end + y - 1) / y), (unsigned)y),
                     dim3(kThreads), 0, stream, p, first_dout, first_a, end);
  return hipGetLastError();
}

}  // namespace fp8
