// ffn_device.h -- what the kernels of the feed-forward block and of MXFP4 share.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

// the host pass sees the kernels' stubs alone
#if !defined(__HIP_DEVICE_COMPILE__)
#pragma clang diagnostic ignored "-Wunused-function"
#pragma clang diagnostic ignored "-Wunneeded-internal-declaration"
#endif

namespace ffn {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 h16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef __attribute__((address_space(3))) uint8_t* lds_bytes;
typedef __attribute__((address_space(3))) u32x2* lds_u32x2;
typedef __attribute__((address_space(3))) u32x4* lds_u32x4;
typedef __attribute__((address_space(3))) f32x4* lds_f32x4;
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

constexpr int kBufferFlags = 0x00020000;  // raw buffer resource, dword 3
constexpr uint32_t kOut = 0x80000000u;    // an offset past every buffer: reads 0

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <int N>
__device__ __forceinline__ void wait_vm() {
  // vmcnt[3:0] | expcnt[6:4] | lgkmcnt[11:8] | vmcnt_hi[15:14]
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0xC07F); }

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// 1 / (1 + e^-g) by the hardware's 2^x and reciprocal: within 2^-19 of itself
// for |g| < 16, beyond that by |g| 2^-23, far below the roundings that follow;
// 0 below -87.3, where it would be subnormal. (Rounding g log2(e) and the
// constant in it give 1.23 |g| 2^-24, the two instructions and the sum 5 times
// 2^-24; over all g the most is 16.5 times 2^-24 below 16, 30.9 below 32 and 60.2
// below 64.)
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-g));
}

// The e8m0 byte of a block from its largest exponent field (fp32's or bf16's):
// two less, at least 0; 255 for infinities and NaN.
__device__ __forceinline__ uint32_t mx_scale(uint32_t exponent) {
  return exponent == 255 ? 255u : exponent < 2 ? 0u : exponent - 2;
}
// The byte as the scale operand of the fp4 conversions: they divide by the
// power of two of its exponent field alone (0: 2^-127), round to nearest even
// and saturate; checked over all bytes, borders included.
__device__ __forceinline__ float mx_unit(uint32_t scale) {
  return __builtin_bit_cast(float, scale << 23);
}

// f(0), ..., f(N - 1), each a constant
template <typename F, int... I>
__device__ __forceinline__ void each(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
  each(f, std::make_integer_sequence<int, N>{});
}

// The tile of this work-group. Work-group i runs on XCD i % 8: each XCD takes
// a run of consecutive tiles, and tiles run through groups of 8 row tiles, so
// that the tiles an XCD holds at one time share rows of A and of B in its L2.
struct TileId {
  int64_t m, n;
};
__device__ __forceinline__ TileId tile_of(int64_t id, int64_t tm, int64_t tn) {
  const int64_t total = tm * tn;
  const int64_t per = total / 8, rest = total % 8;
  const int64_t x = id % 8, i = id / 8;
  const int64_t t = x * per + (x < rest ? x : rest) + i;
  const int64_t group = 8 * tn, g = t / group;
  const int64_t h = tm - g * 8 < 8 ? tm - g * 8 : 8;
  return TileId{g * 8 + (t - g * group) % h, (t - g * group) / h};
}

#if defined(__HIP_DEVICE_COMPILE__)
__device__ __forceinline__ f32x4 mfma(const u32x4& n, const u32x4& m, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, n),
                                                 __builtin_bit_cast(bf16x8, m), c, 0, 0, 0);
}
template <int SN, int SM>
__device__ __forceinline__ f32x4 mfma_mx(const u32x4& n, const u32x4& m, const f32x4& c,
                                         uint32_t sn, uint32_t sm) {
  const i32x8 a = {(int)n[0], (int)n[1], (int)n[2], (int)n[3]};
  const i32x8 b = {(int)m[0], (int)m[1], (int)m[2], (int)m[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, SN, (int)sn, SM,
                                                          (int)sm);
}

#endif

}  // namespace
}  // namespace ffn
