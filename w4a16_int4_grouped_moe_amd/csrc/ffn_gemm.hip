// ffn_gemm.hip -- the matrix products of the feed-forward block and of MXFP4
// (gfx950): D[m, n] = sum_k A(m, k) B(n, k) in fp32, with the block's SwiGLU,
// its gradient or the MXFP4 quantisation of its result in the epilogue.
//
// One skeleton for bf16 and MXFP4. K advances in stages of 128 bytes of a
// row: 64 bf16 or 256 e2m1 values. A lane feeds v_mfma_f32_16x16x32_bf16 and
// v_mfma_scale_f32_16x16x128_f8f6f4 the same 16 bytes at the same cadence
// (16 cycles), so tiles, LDS layout and copies are the same bytes and MXFP4
// does four times the operations with them.
//
// Operands. A bf16 operand is K contiguous (KC) or row contiguous (RC: what
// the gradients read along its other axis); both go from memory into LDS by
// buffer loads with an LDS destination, in whole 128-byte lines, and out of
// range reads zeros (rows past the end, the last stage's missing k).
//   KC: row r holds eight 16-byte pieces, piece c at slot c ^ ((r >> 1) & 7):
//       16 rows at one piece are 16 distinct bank groups of ds_read_b128.
//   RC: k-row k holds 32-byte chunks (16 rows of the operand), chunk c at slot
//       c ^ g(k); ds_read_b64_tr_b16 transposes 4 k x 16 rows per 16 lanes, and
//       g spreads the eight k-rows that 32 lanes read over all 64 banks.
// The MFMA's first operand is B, its second A: a lane then holds four
// consecutive columns n of one row m, which is how outputs are stored.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ffn_internal.h"

namespace ffn {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

constexpr int kBufferFlags = 0x00020000;  // raw buffer resource, dword 3
constexpr uint32_t kOut = 0x80000000u;    // an offset past every buffer: reads 0
constexpr int kRow = 128;                 // bytes of a KC row per stage

enum Kind { KC = 0, RC = 1 };

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <int N>
__device__ __forceinline__ void wait_vm() {
  // vmcnt[3:0] | expcnt[6:4] | lgkmcnt[11:8] | vmcnt_hi[15:14]
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0xC07F); }

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

// 16 lanes address 4 x 16 16-bit values, four neighbouring lanes a row of 16;
// lane i receives column i, row j in element j.
__device__ __forceinline__ s16x4 read_transposed(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p);
}

// One half tile of an operand: HR rows x one stage, copied by NW waves.
template <Kind KIND, int HR, int NW>
struct Half {
  static constexpr int kBytes = HR * kRow;
  static constexpr int kPer = kBytes / 1024 / NW;  // 1 KB copies per wave
  static_assert(kPer >= 2 && kPer % 2 == 0, "copies come in pairs of row groups");
  const uint8_t* base;
  int64_t ld;
  int64_t kleft;    // KC: bytes of a row; RC: k-rows
  int32_t records;  // KC: bytes that may be read; RC: bytes of a k-row
  uint32_t off[kPer];
  int32_t piece;    // KC: byte of this lane's piece in even copies (odd ones: ^ 64)

  // rows [row0, row0 + HR) of an operand of `rows` rows; K: bytes per row (KC) or k-rows (RC)
  __device__ __forceinline__ void init(const void* ptr, int64_t row0, int64_t rows, int64_t ld_,
                                       int64_t K, int wave, int lane) {
    ld = ld_;
    kleft = K;
    const int64_t left = rows - row0;
    const int valid = left <= 0 ? 0 : left < HR ? (int)left : HR;
    if constexpr (KIND == KC) {
      base = (const uint8_t*)ptr + (valid ? row0 * ld : 0);
      records = valid ? (int32_t)((valid - 1) * ld + K) : 0;
      piece = ((lane & 7) ^ (lane >> 4)) * 16;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int r = 8 * (wave * kPer + j) + (lane >> 3);
        off[j] = r < valid ? (uint32_t)(r * ld) + (piece ^ ((j & 1) * 64)) : kOut;
      }
    } else {
      base = (const uint8_t*)ptr + (valid ? row0 * 2 : 0);
      records = 2 * valid;
      constexpr int lanes = HR / 8;  // lanes per k-row
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int k = (64 / lanes) * (wave * kPer + j) + lane / lanes;
        const int s = lane % lanes;
        const int col = (((s >> 1) ^ spread(k)) << 4) + ((s & 1) << 3);
        off[j] = col < valid ? (uint32_t)(k * ld) + 2 * col : kOut;
      }
    }
  }

  // where RC chunk c of k-row k lies: slot c ^ spread(k)
  static __device__ __forceinline__ int spread(int k) {
    return HR == 128 ? (k & 3) | ((k >> 1) & 4) : ((k >> 1) & 1) | ((k >> 2) & 2);
  }

  __device__ __forceinline__ void copy(uint8_t* slot, int64_t stage, int wave) const {
    if constexpr (KIND == KC) {
      const __amdgpu_buffer_rsrc_t res =
          __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, records, kBufferFlags);
      const int64_t k0 = stage * kRow;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const bool in = k0 + (piece ^ ((j & 1) * 64)) < kleft;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (lds_ptr)(slot + (wave * kPer + j) * 1024),
                                                 16, in ? off[j] + (uint32_t)k0 : kOut, 0, 0, 0);
      }
    } else {
      const int64_t left = kleft - stage * 64;
      const int32_t n =
          left <= 0 ? 0 : (int32_t)(((left < 64 ? left : 64) - 1) * ld) + records;
      const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(base + (left > 0 ? stage * 64 * ld : 0)), 0, records ? n : 0, kBufferFlags);
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (lds_ptr)(slot + (wave * kPer + j) * 1024),
                                                 16, off[j], 0, 0, 0);
    }
  }
};

// A wave's fragments of a half tile: F sub-tiles of 16 rows from `first`, for
// the stage's two MFMA steps. Lane (r = lane % 16, q = lane / 16) holds row r's
// k = 8 q .. 8 q + 7 of a step (bf16), or its 32-value block 2 q + step (MXFP4:
// a lane's two scale bytes of a stage are then neighbours).
template <Kind KIND, int HR, int F, bool MX>
struct Frags {
  u32x4 v[2][F];
  static __device__ __forceinline__ int lane_base(int lane) {
    const int q = lane >> 4;
    return (lane & 15) * kRow + (((MX ? 2 * q : q) ^ ((lane >> 1) & 7)) * 16);
  }
  __device__ __forceinline__ void read(const uint8_t* slot, int first, int lane) {
    if constexpr (KIND == KC) {
      const int b = lane_base(lane) + first * kRow;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < F; ++i)
          v[s][i] = *(const u32x4*)(slot + (b ^ (s * (MX ? 16 : 64))) + i * 16 * kRow);
    } else {
      const int q = lane >> 4, j = (lane >> 2) & 3;
      const int x = Half<RC, HR, HR / 16>::spread(8 * q + j);
      const uint8_t* b = slot + (8 * q + j) * (2 * HR) + (lane & 3) * 8;
#pragma unroll
      for (int i = 0; i < F; ++i) {
        const uint8_t* c = b + (((first >> 4) + i) ^ x) * 32;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const s16x4 lo = read_transposed(c + s * 32 * (2 * HR));
          const s16x4 hi = read_transposed(c + (s * 32 + 4) * (2 * HR));
          const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
          v[s][i] = u32x4{l2[0], l2[1], h2[0], h2[1]};
        }
      }
    }
  }
};

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

// Quantises one block of 32 values of which this lane holds 2 x 4 and the
// lanes 16, 32 and 48 away the rest; returns the two groups' codes (16 bits
// each) and the block's scale byte.
__device__ __forceinline__ uint32_t mx_quantize8(const float* v, uint32_t* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu;
    top = b > top ? b : top;
  }
  const uint32_t o1 = __shfl_xor(top, 16);
  top = o1 > top ? o1 : top;
  const uint32_t o2 = __shfl_xor(top, 32);
  top = o2 > top ? o2 : top;
  // e8m0 byte: the exponent field less 2 (subnormal fp32 maxima: 0)
  const int e = (int)(top >> 23);
  const bool bad = e == 255;
  const int s = e < 2 ? 0 : e - 2;
  *scale = bad ? 255u : (uint32_t)s;
  uint32_t c = 0;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = bad ? 0.f : ldexpf(v[4 * g + i], 127 - s);
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, y[0], y[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], 1.0f, 1);
    c |= (w & 0xffffu) << (16 * g);
  }
  return c;
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

// Tile of 128 x (2 x 64): four waves (2 x 2) of 64 rows x (2 x 32) columns.
// Two work-groups share a CU and cover each other's waits.
template <Kind KA, Kind KB, bool MX, Epilogue EPI>
__global__ __launch_bounds__(256, 2) void tile_kernel(const Product p) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass needs the stub alone
  constexpr int NW = 4, HRA = 128, HRB = 64, FA = 4, FB = 2;
  constexpr bool kPaired = EPI == kSwiglu || EPI == kSwigluMx;  // B half 1: the up columns
  constexpr int kCols = kPaired ? HRB : 2 * HRB;                // output columns
  typedef Half<KA, HRA, NW> HA;
  typedef Half<KB, HRB, NW> HB;
  __shared__ __attribute__((aligned(1024))) uint8_t sa0[HA::kBytes], sa1[HA::kBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sb00[HB::kBytes], sb01[HB::kBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sb10[HB::kBytes], sb11[HB::kBytes];
  // MXFP4 scales of a stage: per operand row 8 bytes, see store_scales
  __shared__ __attribute__((aligned(16))) uint8_t ss[2][MX ? (HRA + 2 * HRB) * 8 : 8];

  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t tm = (p.M + HRA - 1) / HRA, tn = (p.N + kCols - 1) / kCols;
  const TileId t = tile_of(blockIdx.x, tm, tn);
  const int64_t m0 = t.m * HRA, n0 = t.n * kCols;

  HA a;
  HB b0, b1;
  const int64_t Kext = KA == KC ? (MX ? p.K / 2 : 2 * p.K) : p.K;
  const int64_t Kextb = KB == KC ? (MX ? p.K / 2 : 2 * p.K) : p.K;
  a.init(p.a, m0, p.M, p.lda, Kext, wave, lane);
  b0.init(p.b, n0, p.N, p.ldb, Kextb, wave, lane);
  if (kPaired)
    b1.init((const uint8_t*)p.b + p.N * p.ldb, n0, p.N, p.ldb, Kextb, wave, lane);
  else
    b1.init(p.b, n0 + HRB, p.N, p.ldb, Kextb, wave, lane);
  const int64_t stages = (p.K + (MX ? 255 : 63)) / (MX ? 256 : 64);

  // MXFP4: thread i keeps the eight scale bytes of tile row i (A's 128 rows,
  // then B's 2 x 64) and stage; bytes past K stand for 1 (their codes are 0).
  const uint8_t* srow = nullptr;
  const int64_t nblocks = p.K / 32;
  if constexpr (MX) {
    const int i = threadIdx.x;
    if (i < HRA) {
      if (m0 + i < p.M) srow = p.a_scales + (m0 + i) * nblocks;
    } else {
      const int half = (i - HRA) / HRB, r = (i - HRA) % HRB;
      const int64_t n = n0 + r + (kPaired ? 0 : half * HRB);
      if (n < p.N) srow = p.b_scales + (n + (kPaired ? half * (int64_t)p.N : 0)) * nblocks;
    }
  }
  auto load_scales = [&](int64_t stage, uint32_t* v) {
    v[0] = v[1] = 0x7f7f7f7fu;
    if (!srow) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t blk = stage * 8 + j;
      const uint32_t byte = blk < nblocks ? srow[blk] : 127u;
      v[j / 4] = (v[j / 4] & ~(0xffu << (8 * (j & 3)))) | (byte << (8 * (j & 3)));
    }
  };
  // the 16-row sub-tiles of a wave's half lie together: lane (r, q) finds its
  // two bytes (blocks 2 q, 2 q + 1) of sub-tile i at ((first + 0) * 8 + r * ..)
  auto store_scales = [&](int buf, const uint32_t* v) {
    const int i = threadIdx.x;
    int base, sub, n;
    if (i < HRA) {
      base = (i / 64) * 64, sub = (i % 64) / 16, n = FA;
    } else {
      base = HRA + ((i - HRA) / 32) * 32, sub = ((i - HRA) % 32) / 16, n = FB;
    }
    uint8_t* d = ss[buf] + base * 8;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *(uint16_t*)(d + (((i & 15) * 4 + q) * n + sub) * 2) = (uint16_t)(v[q / 2] >> (16 * (q & 1)));
  };

  f32x4 acc[2][FA][FB];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) acc[h][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  uint32_t sc[2];
  if constexpr (MX) load_scales(0, sc);
  a.copy(sa0, 0, wave);
  b0.copy(sb00, 0, wave);
  b1.copy(sb10, 0, wave);

  auto step = [&](int64_t s, auto parity) {
    constexpr int cur = decltype(parity)::value;
    const uint8_t* a_now = cur ? sa1 : sa0;
    const uint8_t* b0_now = cur ? sb01 : sb00;
    const uint8_t* b1_now = cur ? sb11 : sb10;
    if constexpr (MX) store_scales(cur, sc);
    wait_vm<0>();
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    a.copy(cur ? sa0 : sa1, s + 1, wave);
    b0.copy(cur ? sb00 : sb01, s + 1, wave);
    b1.copy(cur ? sb10 : sb11, s + 1, wave);
    if constexpr (MX) load_scales(s + 1, sc);
    __builtin_amdgcn_sched_barrier(0);
    Frags<KA, HRA, FA, MX> fa;
    Frags<KB, HRB, FB, MX> fb0, fb1;
    fa.read(a_now, wm * 64, lane);
    fb0.read(b0_now, wn * 32, lane);
    fb1.read(b1_now, wn * 32, lane);
    if constexpr (MX) {
      const int at = (lane & 15) * 4 + (lane >> 4);
      const u32x2 sm = *(const u32x2*)(ss[cur] + wm * 64 * 8 + at * 8);
      const uint32_t sn0 = *(const uint32_t*)(ss[cur] + (HRA + wn * 32) * 8 + at * 4);
      const uint32_t sn1 = *(const uint32_t*)(ss[cur] + (HRA + HRB + wn * 32) * 8 + at * 4);
#define FFN_MX(h, fb, sn, st, i, j)                                                          \
  acc[h][i][j] = mfma_mx<(j & 1) * 2 + st, (i & 1) * 2 + st>(fb.v[st][j], fa.v[st][i],         \
                                                             acc[h][i][j], sn, sm[i / 2]);
#define FFN_MX_I(st, i)             \
  FFN_MX(0, fb0, sn0, st, i, 0)     \
  FFN_MX(0, fb0, sn0, st, i, 1)     \
  FFN_MX(1, fb1, sn1, st, i, 0)     \
  FFN_MX(1, fb1, sn1, st, i, 1)
      FFN_MX_I(0, 0) FFN_MX_I(0, 1) FFN_MX_I(0, 2) FFN_MX_I(0, 3)
      FFN_MX_I(1, 0) FFN_MX_I(1, 1) FFN_MX_I(1, 2) FFN_MX_I(1, 3)
#undef FFN_MX_I
#undef FFN_MX
    } else {
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int i = 0; i < FA; ++i)
#pragma unroll
          for (int j = 0; j < FB; ++j) {
            acc[0][i][j] = mfma(fb0.v[st][j], fa.v[st][i], acc[0][i][j]);
            acc[1][i][j] = mfma(fb1.v[st][j], fa.v[st][i], acc[1][i][j]);
          }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  int64_t s = 0;
  for (; s + 1 < stages; s += 2) {
    step(s, std::integral_constant<int, 0>{});
    step(s + 1, std::integral_constant<int, 1>{});
  }
  if (s < stages) step(s, std::integral_constant<int, 0>{});
  wait_vm<0>();  // the copies past the last stage (zeros) land before the LDS is given up

  // epilogue: lane holds columns nq .. nq + 3 of row m
  const int64_t N = p.N;
#pragma unroll
  for (int i = 0; i < FA; ++i) {
    const int64_t m = m0 + wm * 64 + i * 16 + (lane & 15);
    if constexpr (EPI == kSwigluMx) {
      float h[8];
#pragma unroll
      for (int j = 0; j < FB; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float g = acc[0][i][j][r];
          h[4 * j + r] = g * sigmoid(g) * acc[1][i][j][r];
        }
      uint32_t scale;
      const uint32_t c = mx_quantize8(h, &scale);
      const int64_t nb = n0 + wn * 32;  // the block's first column; N is a multiple of 32
      if (m < p.M && nb < N) {
        const int q = lane >> 4;
        uint8_t* codes = (uint8_t*)p.out + m * (N / 2) + nb / 2;
        *(uint16_t*)(codes + 2 * q) = (uint16_t)c;
        *(uint16_t*)(codes + 8 + 2 * q) = (uint16_t)(c >> 16);
        if (q == 0) ((uint8_t*)p.aux)[m * (N / 32) + nb / 32] = (uint8_t)scale;
      }
      continue;
    }
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      const int64_t nq = n0 + wn * 32 + j * 16 + (lane >> 4) * 4;
      if (m >= p.M) continue;
      if constexpr (EPI == kSwiglu) {
        if (nq >= N) continue;
        float h[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float g = acc[0][i][j][r];
          h[r] = g * sigmoid(g) * acc[1][i][j][r];
        }
        *(u32x2*)((uint16_t*)p.out + m * N + nq) = u32x2{pack2(h[0], h[1]), pack2(h[2], h[3])};
        if (p.aux) {
          float* gu = (float*)p.aux + m * 2 * N + nq;
          *(f32x4*)gu = acc[0][i][j];
          *(f32x4*)(gu + N) = acc[1][i][j];
        }
      } else {
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
          const int64_t n = nq + hb * HRB;
          if (n >= N) continue;
          const f32x4 v = acc[hb][i][j];
          if constexpr (EPI == kStoreF32) {
            *(f32x4*)((float*)p.out + m * N + n) = v;
          } else if constexpr (EPI == kStoreBf16) {
            *(u32x2*)((uint16_t*)p.out + m * N + n) =
                u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
          } else {
            const float* gu = (const float*)p.aux + m * 2 * N + n;
            const f32x4 g = *(const f32x4*)gu, u = *(const f32x4*)(gu + N);
            float dg[4], du[4], h[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float sg = sigmoid(g[r]);
              du[r] = v[r] * g[r] * sg;
              dg[r] = v[r] * u[r] * sg * (1.0f + g[r] * (1.0f - sg));
              h[r] = g[r] * sg * u[r];
            }
            uint16_t* d = (uint16_t*)p.out + m * 2 * N + n;
            *(u32x2*)d = u32x2{pack2(dg[0], dg[1]), pack2(dg[2], dg[3])};
            *(u32x2*)(d + N) = u32x2{pack2(du[0], du[1]), pack2(du[2], du[3])};
            *(u32x2*)((uint16_t*)p.out2 + m * N + n) =
                u32x2{pack2(h[0], h[1]), pack2(h[2], h[3])};
          }
        }
      }
    }
  }
#endif
}

template <Kind KA, Kind KB, bool MX, Epilogue EPI>
hipError_t launch(const Product& p, hipStream_t stream) {
  const int64_t cols = EPI == kSwiglu || EPI == kSwigluMx ? 64 : 128;
  const int64_t tiles = ((p.M + 127) / 128) * ((p.N + cols - 1) / cols);
  if (tiles == 0) return hipSuccess;
  if (tiles > 0x7fffffff) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((tile_kernel<KA, KB, MX, EPI>), dim3((unsigned)tiles), dim3(256), 0, stream,
                     p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_product(Layout layout, Epilogue epilogue, const Product& p,
                          hipStream_t stream) {
  if (layout == kNT && epilogue == kSwiglu) return launch<KC, KC, false, kSwiglu>(p, stream);
  if (layout == kNT && epilogue == kStoreBf16)
    return launch<KC, KC, false, kStoreBf16>(p, stream);
  if (layout == kNN && epilogue == kSwigluGrad)
    return launch<KC, RC, false, kSwigluGrad>(p, stream);
  if (layout == kNN && epilogue == kStoreBf16)
    return launch<KC, RC, false, kStoreBf16>(p, stream);
  if (layout == kTN && epilogue == kStoreBf16)
    return launch<RC, RC, false, kStoreBf16>(p, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_product_mx(Epilogue epilogue, const Product& p, hipStream_t stream) {
  if (epilogue == kStoreBf16) return launch<KC, KC, true, kStoreBf16>(p, stream);
  if (epilogue == kStoreF32) return launch<KC, KC, true, kStoreF32>(p, stream);
  if (epilogue == kSwigluMx) return launch<KC, KC, true, kSwigluMx>(p, stream);
  return hipErrorInvalidValue;
}

}  // namespace ffn
