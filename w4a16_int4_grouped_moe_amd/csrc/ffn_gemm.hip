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

#include <utility>

#include "ffn_device.h"
#include "ffn_internal.h"

namespace ffn {
namespace {

constexpr int kRow = 128;  // bytes of a KC row per stage

enum Kind { KC = 0, RC = 1 };

// 16 lanes address 4 x 16 16-bit values, four neighbouring lanes a row of 16;
// lane i receives column i, row j in element j.
__device__ __forceinline__ s16x4 read_transposed(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p);
}

// Where RC chunk c of k-row k of a half tile of HR rows lies: slot c ^ spread(k).
template <int HR>
__device__ __forceinline__ int spread(int k) {
  return HR == 128 ? (k & 3) | ((k >> 1) & 4) : ((k >> 1) & 1) | ((k >> 2) & 2);
}

// What a lane copies of a half tile (HR rows x one stage, 1 KB a copy, NW
// waves): offsets from the half's base, the same for every half of an operand.
template <Kind KIND, int HR, int NW>
struct Lane {
  static constexpr int kPer = HR * kRow / 1024 / NW;  // copies per wave
  static_assert(kPer >= 2 && kPer % 2 == 0, "copies come in pairs of row groups");
  uint32_t off[kPer];
  int piece;  // KC: byte of this lane's piece in even copies (odd ones: ^ 64)

  __device__ __forceinline__ void init(int64_t ld, int wave, int lane) {
    piece = ((lane & 7) ^ (lane >> 4)) * 16;
    constexpr int lanes = HR / 8;  // RC: lanes per k-row
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if constexpr (KIND == KC) {
        const int r = 8 * (wave * kPer + j) + (lane >> 3);
        off[j] = (uint32_t)(r * ld) + (piece ^ ((j & 1) * 64));
      } else {
        const int k = (64 / lanes) * (wave * kPer + j) + lane / lanes, c = lane % lanes;
        off[j] = (uint32_t)(k * ld) + (((c >> 1) ^ spread<HR>(k)) << 5) + ((c & 1) << 4);
      }
    }
  }
};

// One half tile of an operand. A read past the operand's end gives zeros (its
// resource ends there); rows past the last one (KC: further than the end; RC:
// the next k-row's data) only reach sums that are not stored.
template <Kind KIND, int HR, int NW>
struct Half {
  static constexpr int kBytes = HR * kRow;
  static constexpr int kPer = Lane<KIND, HR, NW>::kPer;
  const uint8_t* base;
  int64_t ld;
  int64_t kleft;    // KC: bytes of a row (fits 32 bits); RC: k-rows
  int32_t records;  // KC: bytes that may be read; RC: bytes of a k-row

  // rows [row0, row0 + HR) of an operand of `rows` rows; K: bytes per row (KC) or k-rows (RC)
  __device__ __forceinline__ void init(const void* ptr, int64_t row0, int64_t rows, int64_t ld_,
                                       int64_t K) {
    ld = ld_;
    kleft = K;
    const int64_t left = rows - row0;
    const int valid = left <= 0 ? 0 : left < HR ? (int)left : HR;
    base = (const uint8_t*)ptr + (valid ? row0 * (KIND == KC ? ld : 2) : 0);
    if constexpr (KIND == KC)
      records = valid ? (int32_t)((valid - 1) * ld + K) : 0;
    else
      records = 2 * valid;
  }

  __device__ __forceinline__ void copy(uint8_t* slot, int stage, int wave,
                                       const Lane<KIND, HR, NW>& at) const {
    uint8_t* dst = slot + wave * (kPer * 1024);
    if constexpr (KIND == KC) {
      const __amdgpu_buffer_rsrc_t res =
          __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, records, kBufferFlags);
      const int k0 = stage * kRow, end = (int)kleft - k0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const bool in = (at.piece ^ ((j & 1) * 64)) < end;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (lds_ptr)(dst + j * 1024), 16,
                                                 in ? at.off[j] + (uint32_t)k0 : kOut, 0, 0, 0);
      }
    } else {
      const int64_t left = kleft - (int64_t)stage * 64;
      const int32_t n =
          left <= 0 ? 0 : (int32_t)(((left < 64 ? left : 64) - 1) * ld) + records;
      const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(base + (left > 0 ? (int64_t)stage * 64 * ld : 0)), 0, records ? n : 0,
          kBufferFlags);
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (lds_ptr)(dst + j * 1024), 16, at.off[j],
                                                 0, 0, 0);
    }
  }
};

// A wave's fragments of a half tile: F sub-tiles of 16 rows from `first`, for
// the stage's two MFMA steps. Lane (r = lane % 16, q = lane / 16) holds piece
// 4 step + q of row r: k = 8 q .. 8 q + 7 of the step (bf16), or its block q
// of 32 (MXFP4).
template <Kind KIND, int HR, int F>
struct Frags {
  u32x4 v[2][F];
  static __device__ __forceinline__ int lane_base(int lane) {
    const int q = lane >> 4;
    return (lane & 15) * kRow + ((q ^ ((lane >> 1) & 7)) * 16);
  }
  __device__ __forceinline__ void read(const uint8_t* slot, int first, int lane) {
    if constexpr (KIND == KC) {
      const int b = lane_base(lane) + first * kRow;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < F; ++i)
          v[s][i] = *(const u32x4*)(slot + (b ^ (s * 64)) + i * 16 * kRow);
    } else {
      const int q = lane >> 4, j = (lane >> 2) & 3;
      const int x = spread<HR>(8 * q + j);
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

#if defined(__HIP_DEVICE_COMPILE__)
// The MFMAs of 16 FA rows x 16 FB columns over a stage. MXFP4: sm and sn hold
// the scale bytes of two sub-tiles a word, two steps each (see put_scales).
template <int FA, int FB, int X>
__device__ __forceinline__ void mma_mx(f32x4 (&acc)[FA][FB], const u32x4 (&n)[2][FB],
                                       const u32x4 (&m)[2][FA], uint32_t sn, u32x2 sm) {
  constexpr int st = X / (FA * FB), i = X / FB % FA, j = X % FB;
  acc[i][j] = mfma_mx<(j & 1) * 2 + st, (i & 1) * 2 + st>(n[st][j], m[st][i], acc[i][j], sn,
                                                          sm[i / 2]);
}
template <bool MX, int FA, int FB, int... X>
__device__ __forceinline__ void mma(f32x4 (&acc)[FA][FB], const u32x4 (&n)[2][FB],
                                    const u32x4 (&m)[2][FA], uint32_t sn, u32x2 sm,
                                    std::integer_sequence<int, X...>) {
  static_assert(FA == 4 && FB == 2, "scale words");
  if constexpr (MX) {
    (mma_mx<FA, FB, X>(acc, n, m, sn, sm), ...);
  } else {
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = mfma(n[st][j], m[st][i], acc[i][j]);
  }
  // an MFMA has no side effect: this keeps them on this side of the barrier that follows
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) asm volatile("" : "+v"(acc[i][j]));
}
#endif

// MXFP4 scales of a tile: thread i carries the eight scale bytes (one stage)
// of tile row i, A's rows first, then B's two halves. Rows and stages past the
// end read the last one: their codes are 0 and their sums are not stored.
template <int ROWS_A, int ROWS_B, int GROUP_A, int GROUP_B, int THREADS>
struct Scales {
  static constexpr int kBytes = (ROWS_A + ROWS_B) * 8;
  const uint8_t* row;
  int last;  // the last stage's offset
  u32x2 v;
  static_assert(ROWS_A + ROWS_B == THREADS, "a thread a row");

  __device__ __forceinline__ void init(const Product& p, int64_t m0, int64_t n0, int64_t n1,
                                       int64_t up) {
    last = (int)scale_stride(p.K) - 8;
    const int i = threadIdx.x;
    if (i < ROWS_A) {
      row = p.a_scales + (m0 + i < p.M ? m0 + i : p.M - 1) * (int64_t)(last + 8);
    } else {
      const int half = (i - ROWS_A) / (ROWS_B / 2), r = (i - ROWS_A) % (ROWS_B / 2);
      const int64_t n = (half ? n1 : n0) + r;
      row = p.b_scales + ((n < p.N ? n : p.N - 1) + (half ? up : 0)) * (int64_t)(last + 8);
    }
  }
  __device__ __forceinline__ void load(int stage) {
    v = *(const u32x2*)(row + (stage * 8 < last ? stage * 8 : last));
  }
  // into LDS in the order the fragments read: a wave's GROUP rows of a half lie
  // together, and lane (r, q)'s bytes (blocks q and 4 + q: one of each step) of
  // its sub-tiles are neighbours
  __device__ __forceinline__ void put(uint8_t* lds) const {
    const int i = threadIdx.x;
    const bool b = i >= ROWS_A;
    const int first = b ? ROWS_A + (i - ROWS_A) / GROUP_B * GROUP_B : i / GROUP_A * GROUP_A;
    const int n = (b ? GROUP_B : GROUP_A) / 16, sub = (i - first) / 16;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *(uint16_t*)(lds + first * 8 + (((i & 15) * 4 + q) * n + sub) * 2) =
          (uint16_t)(((v[0] >> (8 * q)) & 0xff) | (((v[1] >> (8 * q)) & 0xff) << 8));
  }
};

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
  *scale = mx_scale(top >> 23);
  const float unit = mx_unit(*scale);
  uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], unit, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], unit, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], unit, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], unit, 3);
  return *scale == 255 ? 0 : c;
}

// Stores a wave's accumulators: 16 FA rows from m0; columns n0 .. of acc[0], and
// of acc[1] `half` further (or, paired, the up columns of the same h columns).
// A lane holds columns nq .. nq + 3 of row m.
template <Epilogue EPI, int FA, int FB>
__device__ __forceinline__ void finish(const Product& p, int64_t m0, int64_t n0, int half,
                                       const f32x4 (&acc)[2][FA][FB], int lane) {
  const int64_t N = p.N;
#pragma unroll
  for (int i = 0; i < FA; ++i) {
    const int64_t m = m0 + i * 16 + (lane & 15);
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
      const int64_t nb = n0;  // the block's first column; N is a multiple of 32
      if (m < p.M && nb < N) {
        const int q = lane >> 4;
        uint8_t* codes = (uint8_t*)p.out + m * (N / 2) + nb / 2;
        *(uint16_t*)(codes + 2 * q) = (uint16_t)c;
        *(uint16_t*)(codes + 8 + 2 * q) = (uint16_t)(c >> 16);
        if (q == 0) {
          uint8_t* scales = (uint8_t*)p.aux + m * scale_stride(N);
          scales[nb / 32] = (uint8_t)scale;
          if (nb + 32 == N)
            for (int64_t b = N / 32; b < scale_stride(N); ++b) scales[b] = 127;
        }
      }
      continue;
    }
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      const int64_t nq = n0 + j * 16 + (lane >> 4) * 4;
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
          const int64_t n = nq + hb * half;
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
  __shared__ __attribute__((aligned(16))) uint8_t ss[2][MX ? (HRA + 2 * HRB) * 8 : 8];

  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t tm = (p.M + HRA - 1) / HRA, tn = (p.N + kCols - 1) / kCols;
  const TileId t = tile_of(blockIdx.x, tm, tn);
  const int64_t m0 = t.m * HRA, n0 = t.n * kCols;

  HA a;
  HB b0, b1;
  Lane<KA, HRA, NW> la;
  Lane<KB, HRB, NW> lb;
  la.init(p.lda, wave, lane);
  lb.init(p.ldb, wave, lane);
  const int64_t Kext = KA == KC ? (MX ? p.K / 2 : 2 * p.K) : p.K;
  const int64_t Kextb = KB == KC ? (MX ? p.K / 2 : 2 * p.K) : p.K;
  a.init(p.a, m0, p.M, p.lda, Kext);
  b0.init(p.b, n0, p.N, p.ldb, Kextb);
  if (kPaired)
    b1.init((const uint8_t*)p.b + p.N * p.ldb, n0, p.N, p.ldb, Kextb);
  else
    b1.init(p.b, n0 + HRB, p.N, p.ldb, Kextb);
  const int stages = (int)((p.K + (MX ? 255 : 63)) / (MX ? 256 : 64));

  Scales<HRA, 2 * HRB, 64, 32, 256> sc;
  if constexpr (MX)
    sc.init(p, m0, n0, kPaired ? n0 : n0 + HRB, kPaired ? p.N : 0);

  f32x4 acc[2][FA][FB];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) acc[h][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  if constexpr (MX) sc.load(0);
  a.copy(sa0, 0, wave, la);
  b0.copy(sb00, 0, wave, lb);
  b1.copy(sb10, 0, wave, lb);

  auto step = [&](int s, auto parity) {
    constexpr int cur = decltype(parity)::value;
    const uint8_t* a_now = cur ? sa1 : sa0;
    const uint8_t* b0_now = cur ? sb01 : sb00;
    const uint8_t* b1_now = cur ? sb11 : sb10;
    if constexpr (MX) sc.put(ss[cur]);
    wait_vm<0>();
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    a.copy(cur ? sa0 : sa1, s + 1, wave, la);
    b0.copy(cur ? sb00 : sb01, s + 1, wave, lb);
    b1.copy(cur ? sb10 : sb11, s + 1, wave, lb);
    if constexpr (MX) sc.load(s + 1);
    __builtin_amdgcn_sched_barrier(0);
    Frags<KA, HRA, FA> fa;
    Frags<KB, HRB, FB> fb0, fb1;
    fa.read(a_now, wm * 64, lane);
    fb0.read(b0_now, wn * 32, lane);
    fb1.read(b1_now, wn * 32, lane);
    u32x2 sm = {};
    uint32_t sn0 = 0, sn1 = 0;
    if constexpr (MX) {
      const int at = (lane & 15) * 4 + (lane >> 4);
      sm = *(const u32x2*)(ss[cur] + wm * 64 * 8 + at * 8);
      sn0 = *(const uint32_t*)(ss[cur] + (HRA + wn * 32) * 8 + at * 4);
      sn1 = *(const uint32_t*)(ss[cur] + (HRA + HRB + wn * 32) * 8 + at * 4);
    }
    mma<MX>(acc[0], fb0.v, fa.v, sn0, sm, std::make_integer_sequence<int, 2 * FA * FB>{});
    mma<MX>(acc[1], fb1.v, fa.v, sn1, sm, std::make_integer_sequence<int, 2 * FA * FB>{});
    __builtin_amdgcn_sched_barrier(0);
  };
  int s = 0;
  for (; s + 1 < stages; s += 2) {
    step(s, std::integral_constant<int, 0>{});
    step(s + 1, std::integral_constant<int, 1>{});
  }
  if (s < stages) step(s, std::integral_constant<int, 0>{});
  wait_vm<0>();  // the copies past the last stage (zeros) land before the LDS is given up

  finish<EPI, FA, FB>(p, m0 + wm * 64, n0 + wn * 32, HRB, acc, lane);
#endif
}

// Tile of (AH x 128) x (2 x 128), eight waves (2 x 4), each 64 rows of every A
// half x 32 columns of both B halves. A phase is one A half against both B
// halves, 32 MFMAs (512 cycles) a wave. The two waves of a SIMD run half a
// phase apart: one reads fragments and issues copies while the other's MFMAs
// run, with a barrier after each of the two parts; s_setprio keeps the MFMAs
// in front. A half tile is copied into its own place as soon as the phase that
// read it is over.
//
//   AH  buffers  phase  reads      copies                 waits for (at its end)
//   2   2        0      A0 B0 B1   A1 of stage s + 1      A1 of s
//                1      A1         A0 B0 B1 of s + 2      A0 B0 B1 of s + 1
//   1   3        0      A0 B0 B1   all of s + 2           all of s + 1
//
// A part's LDS reads complete before its barrier, so the place is free for the
// copies of the next phase; a copy is waited for before a barrier that every
// wave passes ahead of its reads. Copies have 1.5 (AH = 1: 2) stages to arrive.
template <int AH, Kind KA, Kind KB, bool MX, Epilogue EPI>
__global__ __launch_bounds__(512, 2) void big_tile_kernel(const Product p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NW = 8, HR = 128, FA = 4, FB = 2;
  constexpr bool kPaired = EPI == kSwiglu || EPI == kSwigluMx;
  constexpr int kCols = kPaired ? HR : 2 * HR;
  typedef Half<KA, HR, NW> HA;
  typedef Half<KB, HR, NW> HB;
  constexpr int kCopies = HA::kPer;  // per half tile and wave
  // an object a half tile: the compiler then sees which copies a read has to wait for
  __shared__ __attribute__((aligned(1024))) uint8_t sa0[HA::kBytes], sb0[HB::kBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sc0[HB::kBytes], sa1[HA::kBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sb1[HB::kBytes], sc1[HB::kBytes];
  // AH = 2: the second A halves of the two buffers; AH = 1: the third buffer
  __shared__ __attribute__((aligned(1024))) uint8_t sx0[HA::kBytes], sx1[HB::kBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sx2[AH == 1 ? HB::kBytes : 16];
  __shared__ __attribute__((aligned(16))) uint8_t ss[2][MX ? (AH + 2) * HR * 8 : 8];

  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int64_t tm = (p.M + AH * HR - 1) / (AH * HR), tn = (p.N + kCols - 1) / kCols;
  const TileId t = tile_of(blockIdx.x, tm, tn);
  const int64_t m0 = t.m * (AH * HR), n0 = t.n * kCols;

  HA a0, a1;
  HB b0, b1;
  Lane<KA, HR, NW> la;
  Lane<KB, HR, NW> lb;
  la.init(p.lda, wave, lane);
  lb.init(KA == KC && KB == KC ? p.lda : p.ldb, wave, lane);  // NT: both rows hold K values
  const int64_t ka = KA == KC ? (MX ? p.K / 2 : 2 * p.K) : p.K;
  const int64_t kb = KB == KC ? (MX ? p.K / 2 : 2 * p.K) : p.K;
  a0.init(p.a, m0, p.M, p.lda, ka);
  if constexpr (AH == 2) a1.init(p.a, m0 + HR, p.M, p.lda, ka);
  b0.init(p.b, n0, p.N, p.ldb, kb);
  if (kPaired)
    b1.init((const uint8_t*)p.b + p.N * p.ldb, n0, p.N, p.ldb, kb);
  else
    b1.init(p.b, n0 + HR, p.N, p.ldb, kb);
  const int stages = (int)((p.K + (MX ? 255 : 63)) / (MX ? 256 : 64));

  Scales<AH * HR, 2 * HR, 64, 32, (AH + 2) * HR> sc;
  const bool scaled = MX && threadIdx.x < (AH + 2) * HR;
  if constexpr (MX) {
    if (scaled)
      sc.init(p, m0, n0, kPaired ? n0 : n0 + HR, kPaired ? p.N : 0);
    if (scaled) {
      sc.load(0);
      sc.put(ss[0]);
      sc.load(1);
    }
  }

  f32x4 acc[AH][2][FA][FB];
#pragma unroll
  for (int h = 0; h < 2 * AH; ++h)
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) acc[h / 2][h % 2][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // stages 0 and 1, in the order in which they are waited for
  a0.copy(sa0, 0, wave, la);
  b0.copy(sb0, 0, wave, lb);
  b1.copy(sc0, 0, wave, lb);
  if constexpr (AH == 2) a1.copy(sx0, 0, wave, la);
  a0.copy(sa1, 1, wave, la);
  b0.copy(sb1, 1, wave, lb);
  b1.copy(sc1, 1, wave, lb);
  wait_vm<(AH == 2 ? 4 : 3) * kCopies>();
  wait_lgkm0();
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  if (wave >= NW / 2) __builtin_amdgcn_s_barrier();  // half a phase behind

  Frags<KA, HR, FA> fa;
  Frags<KB, HR, FB> fb0, fb1;
  u32x2 sm = {};
  uint32_t sn0 = 0, sn1 = 0;
  const int at = (lane & 15) * 4 + (lane >> 4);

#define FFN_MEM_DONE                     \
  wait_lgkm0();                          \
  __builtin_amdgcn_sched_barrier(0);     \
  __builtin_amdgcn_s_barrier();          \
  __builtin_amdgcn_sched_barrier(0);     \
  __builtin_amdgcn_s_setprio(1);
#define FFN_MMA_DONE                     \
  __builtin_amdgcn_s_setprio(0);         \
  __builtin_amdgcn_sched_barrier(0);     \
  __builtin_amdgcn_s_barrier();          \
  __builtin_amdgcn_sched_barrier(0);
#define FFN_MMA(ah)                                                                         \
  mma<MX>(acc[ah][0], fb0.v, fa.v, sn0, sm, std::make_integer_sequence<int, 2 * FA * FB>{}); \
  mma<MX>(acc[ah][1], fb1.v, fa.v, sn1, sm, std::make_integer_sequence<int, 2 * FA * FB>{});

  // stage s in buffer `buf`; sbuf: its scales' buffer
  auto step = [&](int s, auto buffer, int sbuf) {
    constexpr int buf = decltype(buffer)::value;
    constexpr int two = (buf + 2) % 3;  // AH = 1: the buffer of stage s + 2
    uint8_t* a_now = buf == 0 ? sa0 : buf == 1 ? sa1 : sx0;
    uint8_t* b0_now = buf == 0 ? sb0 : buf == 1 ? sb1 : sx1;
    uint8_t* b1_now = buf == 0 ? sc0 : buf == 1 ? sc1 : sx2;
    fa.read(a_now, wm * 64, lane);
    fb0.read(b0_now, wn * 32, lane);
    fb1.read(b1_now, wn * 32, lane);
    if constexpr (MX) {
      sm = *(const u32x2*)(ss[sbuf] + wm * 64 * 8 + at * 8);
      sn0 = *(const uint32_t*)(ss[sbuf] + (AH * HR + wn * 32) * 8 + at * 4);
      sn1 = *(const uint32_t*)(ss[sbuf] + (AH * HR + HR + wn * 32) * 8 + at * 4);
    }
    if constexpr (AH == 2) {
      a1.copy(buf ? sx0 : sx1, s + 1, wave, la);
      wait_vm<4 * kCopies>();
      FFN_MEM_DONE
      FFN_MMA(0)
      FFN_MMA_DONE
      fa.read(buf ? sx1 : sx0, wm * 64, lane);
      if constexpr (MX) {
        sm = *(const u32x2*)(ss[sbuf] + (HR + wm * 64) * 8 + at * 8);
        sc.put(ss[sbuf ^ 1]);
        sc.load(s + 2);
      }
      a0.copy(a_now, s + 2, wave, la);
      b0.copy(b0_now, s + 2, wave, lb);
      b1.copy(b1_now, s + 2, wave, lb);
      wait_vm<4 * kCopies>();
      FFN_MEM_DONE
      FFN_MMA(1)
      FFN_MMA_DONE
    } else {
      if constexpr (MX) {
        if (scaled) {
          sc.put(ss[sbuf ^ 1]);
          sc.load(s + 2);
        }
      }
      a0.copy(two == 0 ? sa0 : two == 1 ? sa1 : sx0, s + 2, wave, la);
      b0.copy(two == 0 ? sb0 : two == 1 ? sb1 : sx1, s + 2, wave, lb);
      b1.copy(two == 0 ? sc0 : two == 1 ? sc1 : sx2, s + 2, wave, lb);
      wait_vm<3 * kCopies>();
      FFN_MEM_DONE
      FFN_MMA(0)
      FFN_MMA_DONE
    }
  };
  int s = 0;
  if constexpr (AH == 2) {
    for (; s + 1 < stages; s += 2) {
      step(s, std::integral_constant<int, 0>{}, 0);
      step(s + 1, std::integral_constant<int, 1>{}, 1);
    }
    if (s < stages) step(s, std::integral_constant<int, 0>{}, 0);
  } else {
    for (; s + 2 < stages; s += 3) {
      step(s, std::integral_constant<int, 0>{}, s & 1);
      step(s + 1, std::integral_constant<int, 1>{}, (s + 1) & 1);
      step(s + 2, std::integral_constant<int, 2>{}, s & 1);
    }
    if (s < stages) step(s, std::integral_constant<int, 0>{}, s & 1);
    if (s + 1 < stages) step(s + 1, std::integral_constant<int, 1>{}, (s + 1) & 1);
  }
#undef FFN_MEM_DONE
#undef FFN_MMA_DONE
#undef FFN_MMA
  if (wave < NW / 2) __builtin_amdgcn_s_barrier();
  wait_vm<0>();  // the copies past the last stage (zeros) land before the LDS is given up
#pragma unroll
  for (int h = 0; h < AH; ++h)
    finish<EPI, FA, FB>(p, m0 + h * HR + wm * 64, n0 + wn * 32, HR, acc[h], lane);
#endif
}

template <Kind KA, Kind KB, bool MX, Epilogue EPI>
hipError_t launch(const Product& p, hipStream_t stream) {
  constexpr bool paired = EPI == kSwiglu || EPI == kSwigluMx;
  auto tiles = [&](int64_t rows, int64_t cols) {
    return ((p.M + rows - 1) / rows) * ((p.N + cols - 1) / cols);
  };
  const int64_t small = tiles(128, paired ? 64 : 128);
  if (small == 0) return hipSuccess;
  if (small > 0x7fffff) return hipErrorInvalidConfiguration;
  const int64_t b2 = tiles(256, paired ? 128 : 256), b1 = tiles(128, paired ? 128 : 256);
  // The tile by the time of a stage of K over all rounds of its work-groups on
  // 256 CUs, in quarters of the 256 x 256 tile's 1.45 us: a 128 x 256 tile's
  // stage takes 1.19 us (at 4096 tokens, 7168/2048: d h 133 us against 181 in
  // 128 tiles of 256 x 256; the gate and up product 201 against 163), a round
  // of two 128 x 128 tiles a CU 1.0 to 1.4 us (167 us and 232 us there), of
  // one 0.75 us. Of equals the larger tile.
  auto rounds = [](int64_t n, int64_t at_once) { return (double)((n + at_once - 1) / at_once); };
  const double t2 = 4.0 * rounds(b2, 256), t1 = 3.3 * rounds(b1, 256);
  const double t0 = small <= 256 ? 2.1 : 3.4 * rounds(small, 512);
  if (t2 <= t1 && t2 <= t0)
    hipLaunchKernelGGL((big_tile_kernel<2, KA, KB, MX, EPI>), dim3((unsigned)b2), dim3(512), 0,
                       stream, p);
  else if (t1 <= t0)
    hipLaunchKernelGGL((big_tile_kernel<1, KA, KB, MX, EPI>), dim3((unsigned)b1), dim3(512), 0,
                       stream, p);
  else
    hipLaunchKernelGGL((tile_kernel<KA, KB, MX, EPI>), dim3((unsigned)small), dim3(256), 0,
                       stream, p);
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
