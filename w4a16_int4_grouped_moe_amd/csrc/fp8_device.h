// fp8_device.h -- what the FP8 kernels share: e4m3 codes under power-of-two scales.
#pragma once
#include "../../include/moe_ffn.h"
#include "ffn_device.h"
#include "fp8_internal.h"

namespace fp8 {
namespace {

using namespace ffn;

constexpr int kRow = kBlock;  // bytes of a row per stage

// The exponent field of a block's scale from the largest magnitude's bits: 448 is
// 1.75 * 2^8, so a mantissa up to 1.75 leaves 2^-8 of its power of two, a larger one
// 2^-7; at least the least normal, and 1 for a block of zeros. Infinities and NaN: 255.
__device__ __forceinline__ uint32_t scale_field(uint32_t top) {
  if (top >= 0x7f800000u) return 255;
  if (top == 0) return 127;
  const uint32_t e = (top + 0x1fffffu) >> 23;
  return e > 8 ? e - 8 : 1;
}
__device__ __forceinline__ float scale_value(uint32_t field) {
  return field == 255 ? __builtin_nanf("") : __builtin_bit_cast(float, field << 23);
}
// 1 / scale (field 1 .. 247), exact; 0 for NaN, under which codes are 0
__device__ __forceinline__ float scale_inverse(uint32_t field) {
  return field == 255 ? 0.f : __builtin_bit_cast(float, (254 - field) << 23);
}

#if defined(__HIP_DEVICE_COMPILE__)
// Four values times `inverse` as e4m3. At most 448 in magnitude, so nothing saturates; a value
// that the multiplication rounds is below 2^-126, and its code 0 either way. An infinity or a
// NaN has inverse 0 and gives NaN codes: cleared by the caller.
__device__ __forceinline__ uint32_t pack4(const float* v, float inverse) {
  int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inverse, v[1] * inverse, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inverse, v[3] * inverse, c, true);
}
#endif

__device__ __forceinline__ uint32_t magnitude(float v) {
  return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Eight values of x from `unit` eights
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
__device__ __forceinline__ uint32_t top8(const float* v) {
  uint32_t top = magnitude(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) top = larger(top, magnitude(v[i]));
  return top;
}
template <int CTRL>
__device__ __forceinline__ uint32_t with_lane(uint32_t v) {
  return larger(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
// The largest of 16 neighbouring lanes
__device__ __forceinline__ uint32_t top_of_16(uint32_t v) {
  v = with_lane<0xB1>(v);   // lane ^ 1
  v = with_lane<0x4E>(v);   // lane ^ 2
  v = with_lane<0x141>(v);  // mirrored in eights
  return with_lane<0x140>(v);  // mirrored in sixteens
}

__device__ __forceinline__ u32x2 codes8(const float* v, uint32_t field) {
#if defined(__HIP_DEVICE_COMPILE__)
  const float inverse = scale_inverse(field);
  const u32x2 c = {pack4(v, inverse), pack4(v + 4, inverse)};
  return field == 255 ? u32x2{0, 0} : c;
#else
  return u32x2{};
#endif
}

typedef __attribute__((address_space(3))) float* lds_f32;
typedef __attribute__((address_space(3))) int32_t* lds_i32;
typedef const __attribute__((address_space(4))) float* const_f32;

// A wave's fragments of F sub-tiles of 16 rows from `first`
template <int F>
struct Frags {
  u32x4 v[F][2];
  __device__ __forceinline__ void read(lds_bytes slot, int first, int lane) {
    const int q = lane >> 4;
    const int b = (lane & 15) * kRow + ((q ^ ((lane >> 1) & 7)) * 16) + first * kRow;
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        v[i][s] = *(lds_u32x4)(slot + (b ^ (s * 64)) + i * 16 * kRow);
  }
};

#if defined(__HIP_DEVICE_COMPILE__)
__device__ __forceinline__ i32x8 join8(const u32x4 (&v)[2]) {
  return i32x8{(int)v[0][0], (int)v[0][1], (int)v[0][2], (int)v[0][3],
               (int)v[1][0], (int)v[1][1], (int)v[1][2], (int)v[1][3]};
}
// a stage's products of 16 x 16, unscaled
__device__ __forceinline__ f32x4 mfma8(const u32x4 (&n)[2], const u32x4 (&m)[2]) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join8(n), join8(m),
                                                          f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0,
                                                          0);
}

// B's scales of the columns that a lane holds: one, or four a sub-tile
template <bool ROWS, int FB>
struct ColumnScales {
  float v[ROWS ? FB : 1][ROWS ? 4 : 1];
  __device__ __forceinline__ void set(float s) {
    if constexpr (!ROWS) v[0][0] = s;
  }
  __device__ __forceinline__ void read(lds_bytes at, int first, int lane) {
    if constexpr (ROWS)
#pragma unroll
      for (int j = 0; j < FB; ++j) {
        const f32x4 s = *(lds_f32x4)(at + (first + 16 * j + 4 * (lane >> 4)) * 4);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[j][r] = s[r];
      }
  }
};

// acc += the stage's products of 16 FA rows x 16 FB columns of H halves of B, with their
// scales. An MFMA's result is used kLag MFMAs later.
template <bool ROWS, int H, int FA, int FB>
__device__ __forceinline__ void mma(f32x4 (&acc)[H][FA][FB], const Frags<FB> (&n)[H],
                                    const Frags<FA>& m, const float (&sa)[FA],
                                    const ColumnScales<ROWS, FB> (&sb)[H]) {
  constexpr int kAll = H * FA * FB, kLag = kAll < 4 ? kAll : 4;
  f32x4 t[kLag];
  each<kAll + kLag>([&](auto index) {
    constexpr int x = decltype(index)::value;
    if constexpr (x >= kLag) {
      constexpr int y = x - kLag, h = y / (FA * FB), i = y / FB % FA, j = y % FB;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[h][i][j][r] = __builtin_fmaf(
            t[y % kLag][r], sa[i] * sb[h].v[ROWS ? j : 0][ROWS ? r : 0], acc[h][i][j][r]);
    }
    if constexpr (x < kAll) t[x % kLag] = mfma8(n[x / (FA * FB)].v[x % FB], m.v[x / FB % FA]);
    __builtin_amdgcn_sched_barrier(0);  // or the compiler moves a result's use up to its MFMA
  });
}

// Two codes of a word as bf16, which holds every e4m3
template <int HALF>
__device__ __forceinline__ uint32_t widen2(uint32_t codes) {
  return __builtin_bit_cast(uint32_t,
                            __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, HALF != 0));
}
// Word W (two codes) of quarter K (eight codes) of a lane's 32, widened
template <int K, int W>
__device__ __forceinline__ uint32_t widen(const u32x4 (&v)[2]) {
  return widen2<W % 2>(v[K / 2][K % 2 * 2 + W / 2]);
}
// Fragments widened to bf16, a quarter of the stage an MFMA operand
template <int F>
struct Wide {
  u32x4 v[F][4];
  __device__ __forceinline__ void set(const Frags<F>& f) {
#pragma unroll
    for (int i = 0; i < F; ++i)
      each<16>([&](auto x) {
        constexpr int k = decltype(x)::value / 4, w = decltype(x)::value % 4;
        v[i][k][w] = widen<k, w>(f.v[i]);
      });
  }
};
// The same with the products summed in fp32 as the matrix units do it for bf16. A is widened on
// the way: beside each MFMA go its share of the next quarter's four conversions and one
// multiply-add of the sub-tiles before.
template <bool ROWS, int H, int FA, int FB>
__device__ __forceinline__ void mma_wide(f32x4 (&acc)[H][FA][FB], const Wide<FB> (&n)[H],
                                         const Frags<FA>& m, const float (&sa)[FA],
                                         const ColumnScales<ROWS, FB> (&sb)[H]) {
  constexpr int C = H * FB, kAll = FA * 4 * C;  // MFMAs: sub-tile row, quarter, column
  f32x4 t[2][C];
  u32x4 now = {}, next = {};
  each<4>([&](auto w) { now[decltype(w)::value] = widen<0, decltype(w)::value>(m.v[0]); });
  const auto add = [&](auto row, auto element) {  // one value of a sub-tile row's sums
    constexpr int i = decltype(row)::value, c = decltype(element)::value / 4;
    constexpr int r = decltype(element)::value % 4, h = c / FB, j = c % FB;
    acc[h][i][j][r] = __builtin_fmaf(
        t[i & 1][c][r], sa[i] * sb[h].v[ROWS ? j : 0][ROWS ? r : 0], acc[h][i][j][r]);
  };
  each<kAll>([&](auto index) {
    constexpr int x = decltype(index)::value, i = x / (4 * C), k = x / C % 4, c = x % C;
    t[i & 1][c] = mfma(n[c / FB].v[c % FB][k], now, k ? t[i & 1][c] : f32x4{0.f, 0.f, 0.f, 0.f});
    if constexpr (i * 4 + k + 1 < FA * 4) {
      constexpr int ni = (i * 4 + k + 1) / 4, nk = (k + 1) % 4;
      each<4 / C>([&](auto w) {
        constexpr int word = c * (4 / C) + decltype(w)::value;
        next[word] = widen<nk, word>(m.v[ni]);
      });
    }
    if constexpr (i > 0)
      add(std::integral_constant<int, i - 1>{}, std::integral_constant<int, x % (4 * C)>{});
    if constexpr (c == C - 1) now = next;
    __builtin_amdgcn_sched_barrier(0);
  });
  each<4 * C>([&](auto e) { add(std::integral_constant<int, FA - 1>{}, e); });
}

// An MFMA has no side effect: this keeps the sums on this side of the barrier that follows
template <int H, int FA, int FB>
__device__ __forceinline__ void hold(f32x4 (&acc)[H][FA][FB]) {
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) asm volatile("" : "+v"(acc[h][i][j]));
}
#endif

}  // namespace
}  // namespace fp8
