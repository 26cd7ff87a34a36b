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

#include "ffn_device.h"
#include "ffn_internal.h"

namespace ffn {
namespace {

constexpr int kRow = 128;  // bytes of a KC row per stage

enum Kind { KC = 0, RC = 1 };

// 16 lanes address 4 x 16 16-bit values, four neighbouring lanes a row of 16;
// lane i receives column i, row j in element j.
__device__ __forceinline__ s16x4 read_transposed(lds_bytes p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p);
}

// Where RC chunk c of k-row k of a half tile of HR rows lies: slot c ^ spread(k).
template <int HR>
__device__ __forceinline__ int spread(int k) {
  return HR == 128 ? (k & 3) | ((k >> 1) & 4)
         : HR == 64 ? ((k >> 1) & 1) | ((k >> 2) & 2)
                    : (k >> 3) & 1;
}

// What a lane copies of a half tile (HR rows x one stage, 1 KB a copy, NW
// waves): offsets from the half's base, the same for every half of an operand.
template <Kind KIND, int HR, int NW>
struct Lane {
  static constexpr int kPer = HR * kRow / 1024 / NW;  // copies per wave
  static_assert(kPer == 1 || kPer % 2 == 0, "a wave's copies start at an even row group, or one each");
  uint32_t off[kPer];
  int piece;  // KC: byte of this lane's piece in even copies (odd ones: ^ 64)

  __device__ __forceinline__ void init(int64_t ld, int wave, int lane) {
    piece = (((lane & 7) ^ (lane >> 4)) * 16) ^ (kPer == 1 ? (wave & 1) * 64 : 0);
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
  int64_t pitch;    // RC: bytes of a stage
  int32_t end;      // KC: bytes of a row; RC: k-rows
  int32_t span;     // RC: bytes from a k-row to the next, 0 where the half has no rows
  int32_t records;  // KC: bytes that may be read; RC: bytes of a k-row

  // rows [row0, row0 + HR) of an operand of `rows` rows; K: bytes per row (KC) or k-rows (RC),
  // of which the first `end` are read
  __device__ __forceinline__ void init(const void* ptr, int64_t row0, int64_t rows, int64_t ld,
                                       int64_t K, int64_t end_) {
    end = (int32_t)end_;
    const int64_t left = rows - row0;
    const int valid = left <= 0 ? 0 : left < HR ? (int)left : HR;
    base = (const uint8_t*)ptr + (valid ? row0 * (KIND == KC ? ld : 2) : 0);
    if constexpr (KIND == KC)
      records = valid ? (int32_t)((valid - 1) * ld + K) : 0;
    else
      records = 2 * valid, span = valid ? (int32_t)ld : 0, pitch = 64 * ld;
  }

  __device__ __forceinline__ void copy(lds_bytes slot, int stage, int wave,
                                       const Lane<KIND, HR, NW>& at) const {
    const lds_bytes dst = slot + wave * (kPer * 1024);
    if constexpr (KIND == KC) {
      const __amdgpu_buffer_rsrc_t res =
          __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, records, kBufferFlags);
      const int k0 = stage * kRow, left = end - k0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const bool in = (at.piece ^ ((j & 1) * 64)) < left;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (lds_ptr)(dst + j * 1024), 16,
                                                 in ? at.off[j] + (uint32_t)k0 : kOut, 0, 0, 0);
      }
    } else {
      // the end of the stage's last k-row; past K (by seven stages at most) below 0. Without a
      // branch, behind which the compiler would no longer know how many copies are in flight.
      const int left = (int)((uint32_t)end - 64u * (uint32_t)stage);
      const int bytes = ((left < 64 ? left : 64) - 1) * span + records;
      const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(base + stage * pitch), 0, bytes < 0 ? 0 : bytes, kBufferFlags);
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
  __device__ __forceinline__ void read(lds_bytes slot, int first, int lane) {
    if constexpr (KIND == KC) {
      const int b = lane_base(lane) + first * kRow;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < F; ++i)
          v[s][i] = *(lds_u32x4)(slot + (b ^ (s * 64)) + i * 16 * kRow);
    } else {
      const int q = lane >> 4, j = (lane >> 2) & 3;
      const int x = spread<HR>(8 * q + j);
      const lds_bytes b = slot + (8 * q + j) * (2 * HR) + (lane & 3) * 8;
#pragma unroll
      for (int i = 0; i < F; ++i) {
        const lds_bytes c = b + (((first >> 4) + i) ^ x) * 32;
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
// the scale bytes of two sub-tiles a word, two steps each (see read_scales).
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
  static_assert(FA <= 4 && FB <= 2, "scale words");
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

// The MXFP4 scales that a wave copies, 8 bytes a row and stage: ROWS rows of a
// tile (or none), so that every wave has one such copy a stage in flight.
template <int ROWS>
struct WaveScales {
  const uint8_t* base;
  int64_t pitch;  // bytes of a stage
  int32_t records, last, lanes, at;
  // rows from row0 of an operand, which is `rows` rows from `first` of a matrix of `all`; at:
  // their place in the LDS object
  __device__ __forceinline__ void init(const uint8_t* scales, int64_t first, int64_t row0,
                                       int64_t rows, int64_t all, int64_t K, int at_, bool any) {
    pitch = 8 * scale_rows(all);
    last = (int)scale_stages(K) - 1;
    const int64_t left = rows - row0;
    records = left <= 0 ? 0 : (int32_t)((left < ROWS ? scale_rows(left) : ROWS) * 8);
    base = scales + (left > 0 ? first + row0 : 0) * 8;
    lanes = any ? ROWS / 2 : 0;
    at = at_;
  }
  __device__ __forceinline__ void copy(lds_bytes slot, int stage, int lane) const {
    const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(base + (stage < last ? stage : last) * pitch), 0, records, kBufferFlags);
    if (lane < lanes)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (lds_ptr)(slot + at), 16, 16 * lane, 0, 0, 0);
  }
};

// A wave's scale operands: lane (r, q) takes bytes q and 4 + q (its blocks of
// the two steps) of row r of each sub-tile; two sub-tiles a word.
template <int F>
__device__ __forceinline__ void read_scales(lds_bytes slot, int first, int lane,
                                            uint32_t* word) {
  const int q = lane >> 4;
  const uint32_t pick = (uint32_t)(q | (4 + q) << 8);
  const lds_bytes at = slot + (first + (lane & 15)) * 8;
#pragma unroll
  for (int i = 0; i < F; i += 2) {
    const u32x2 a = *(lds_u32x2)(at + i * 16 * 8);
    const uint32_t lo = __builtin_amdgcn_perm(a[1], a[0], pick);
    if constexpr (F == 1) {
      word[0] = lo;
      return;
    }
    const u32x2 b = *(lds_u32x2)(at + (i + 1) * 16 * 8);
    const uint32_t hi = __builtin_amdgcn_perm(b[1], b[0], pick);
    word[i / 2] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
  }
}

// The scale byte of h's block from column n of row m; the last block fills its stage.
__device__ __forceinline__ void put_scale(const Product& p, int64_t m, int64_t n, uint32_t scale) {
  uint8_t* dst = (uint8_t*)p.aux + (n / 256 * scale_rows(p.M) + m) * 8;
  const int at = (int)(n / 32) & 7;
  dst[at] = (uint8_t)scale;
  if (n + 32 == p.N)
    for (int i = at + 1; i < 8; ++i) dst[i] = 127;
}

// Four columns from n of row m: `v`, or a gate and an up group. h is rounded to
// bf16 here, once: it is the next product's operand, which the matrix units take in
// 16 bits.
template <Epilogue EPI>
__device__ __forceinline__ void emit(const Product& p, int64_t m, int64_t n, const f32x4& v,
                                     const f32x4& up) {
  const int64_t N = p.N;
  if constexpr (EPI == kStoreF32 || EPI == kPartial) {
    *(f32x4*)((float*)p.out + m * N + n) = v;
  } else if constexpr (EPI == kPartialPaired) {
    float* gu = (float*)p.out + m * 2 * N + n;
    *(f32x4*)gu = v;
    *(f32x4*)(gu + N) = up;
  } else if constexpr (EPI == kStoreBf16 || EPI == kStoreOrSums) {
    if (EPI == kStoreOrSums && p.aux)
      *(f32x4*)((float*)p.aux + m * N + n) = v;
    else
      *(u32x2*)((uint16_t*)p.out + m * N + n) = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
  } else if constexpr (EPI == kSwiglu) {
    float h[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = v[r] * sigmoid(v[r]) * up[r];
    *(u32x2*)((uint16_t*)p.out + m * N + n) = u32x2{pack2(h[0], h[1]), pack2(h[2], h[3])};
    if (p.aux) {
      float* gu = (float*)p.aux + m * 2 * N + n;
      *(f32x4*)gu = v;
      *(f32x4*)(gu + N) = up;
    }
  }
}

// Four columns of dh -> the gradients of g and u, and h: operands of the last
// products, rounded to bf16 once for the matrix units.
__device__ __forceinline__ void emit_grad(const Product& p, int64_t m, int64_t n, const f32x4& v,
                                          const f32x4& g, const f32x4& u) {
  const int64_t N = p.N;
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
  *(u32x2*)((uint16_t*)p.out2 + m * N + n) = u32x2{pack2(h[0], h[1]), pack2(h[2], h[3])};
}
__device__ __forceinline__ void load_gate_up(const Product& p, int64_t m, int64_t n, f32x4& g,
                                             f32x4& u) {
  const float* gu = (const float*)p.aux + m * 2 * (int64_t)p.N + n;
  g = *(const f32x4*)gu;
  u = *(const f32x4*)(gu + p.N);
}

// Four h columns from n of row m, quantised with the seven lanes that hold the
// rest of the block (eight neighbours); lanes that store nothing take part.
__device__ __forceinline__ void emit_mx(const Product& p, int64_t m, int64_t n, const f32x4& g,
                                        const f32x4& u, bool in) {
  float h[4];
  uint32_t top = 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    h[r] = g[r] * sigmoid(g[r]) * u[r];
    const uint32_t b = __builtin_bit_cast(uint32_t, h[r]) & 0x7fffffffu;
    top = b > top ? b : top;
  }
#pragma unroll
  for (int x = 1; x < 8; x *= 2) {
    const uint32_t o = __shfl_xor(top, x);
    top = o > top ? o : top;
  }
  const uint32_t scale = mx_scale(top >> 23);
  const float unit = mx_unit(scale);
  uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, h[0], h[1], unit, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, h[2], h[3], unit, 1);
  if (!in) return;
  ((uint16_t*)p.out)[(m * p.N + n) / 4] = scale == 255 ? 0 : (uint16_t)c;
  if ((n & 31) == 0) put_scale(p, m, n, scale);
}

// A tile leaves through LDS as fp32 rows, so that memory sees whole rows: the
// waves write their accumulators (16-byte piece c of row r at c ^ (r % 16)),
// then each takes ROWS whole rows, a lane four columns of one (paired: of its
// gate and its up columns). COLS: columns of a row in LDS; m0: the row of the
// tile's matrix at `lds`.
template <Epilogue EPI, int ROWS, int COLS>
__device__ __forceinline__ void store_rows(const Product& p, lds_bytes lds, int64_t m0,
                                           int64_t n0, int lane) {
  constexpr bool kPaired = EPI == kSwiglu || EPI == kSwigluMx || EPI == kPartialPaired;
  constexpr int kLanes = COLS / (kPaired ? 8 : 4);  // a row's lanes
  constexpr int kRowsAtOnce = 64 / kLanes, kTurns = ROWS / kRowsAtOnce;
  constexpr int kMost = kPaired ? 4 : 8, kBatch = kTurns < kMost ? kTurns : kMost;
  const int c = lane % kLanes;
  const int64_t n = n0 + 4 * c;
#pragma unroll
  for (int t = 0; t < kTurns; t += kBatch) {
    f32x4 v[kBatch], up[kBatch], g[kBatch];
    if constexpr (EPI == kSwigluGrad) {  // a batch's pre-activations on their way together
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int64_t m = m0 + kRowsAtOnce * (t + k) + lane / kLanes;
        g[k] = up[k] = f32x4{};
        if (m < p.M && n < p.N) load_gate_up(p, m, n, g[k], up[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int x = kRowsAtOnce * (t + k) + lane / kLanes;
      v[k] = *(lds_f32x4)(lds + x * (4 * COLS) + ((c ^ (x & 15)) * 16));
      if constexpr (kPaired)
        up[k] = *(lds_f32x4)(lds + x * (4 * COLS) + (((c + kLanes) ^ (x & 15)) * 16));
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t m = m0 + kRowsAtOnce * (t + k) + lane / kLanes;
      const bool in = m < p.M && n < p.N;
      if constexpr (EPI == kSwigluMx) {
        emit_mx(p, m, n, v[k], up[k], in);
      } else if constexpr (EPI == kSwigluGrad) {
        if (in) emit_grad(p, m, n, v[k], g[k], up[k]);
      } else {
        if (in) emit<EPI>(p, m, n, v[k], up[k]);
      }
    }
  }
}

// A small tile's ring of stages (four of 128 x 128, eight of 64 x 64): an object
// a stage and half, so that the compiler sees which copies a read has to wait
// for. `a` also holds the tile on its way out.
template <int D>
struct Ring {
  lds_bytes a[D], b[D], c[D], s[D];
};
#define FFN_STAGE(i, tile, scales)                                            \
  __shared__ __attribute__((aligned(1024))) uint8_t sa##i[(tile) * kRow];     \
  __shared__ __attribute__((aligned(1024))) uint8_t sb##i[(tile) / 2 * kRow]; \
  __shared__ __attribute__((aligned(1024))) uint8_t sc##i[(tile) / 2 * kRow]; \
  __shared__ __attribute__((aligned(16))) uint8_t ss##i[scales];              \
  ring.a[i] = (lds_bytes)sa##i, ring.b[i] = (lds_bytes)sb##i;                 \
  ring.c[i] = (lds_bytes)sc##i, ring.s[i] = (lds_bytes)ss##i;
#define FFN_STAGES4(tile, scales) \
  FFN_STAGE(0, tile, scales)      \
  FFN_STAGE(1, tile, scales) FFN_STAGE(2, tile, scales) FFN_STAGE(3, tile, scales)
#define FFN_STAGES8(tile, scales) \
  FFN_STAGES4(tile, scales)       \
  FFN_STAGE(4, tile, scales)      \
  FFN_STAGE(5, tile, scales) FFN_STAGE(6, tile, scales) FFN_STAGE(7, tile, scales)

#if defined(__HIP_DEVICE_COMPILE__)
// Tile of TS x (2 x TS / 2), TS = 128 or 64: four waves (2 x 2) of TS / 2 rows x (2
// x TS / 4) columns, for launches that leave CUs idle: a ring of D stages, copied
// D - 1 ahead, and one barrier a stage. The stages from `first`, at most `share`
// of them. 64 x 64 with seven copies under way takes 0.32 us a stage (0.36 row
// contiguous, 0.40 MXFP4) where 128 x 128 with three takes 0.62 (0.70, 0.85) for
// four times the work, its 32 MFMAs a wave being 0.21; 4 to 4.5 us besides, for the
// first copies and the way out. Neither memory nor the matrix units bound it: 333
// tokens' gate and up at 1000/680 (10.5 us) keep the matrix units busy in 10% of
// the cycles; a wave issues in 34% of its cycles, waits for copies, LDS and the
// barrier in 40%, for its turn to issue in 25%. The block on them: 17.0 us with 64
// x 64 tiles, 26.9 with 128 x 128 in shares of K.
template <int TS, Kind KA, Kind KB, bool MX, Epilogue EPI>
__device__ __forceinline__ void tile_body(const Product& p, const Ring<512 / TS>& at, int64_t id,
                                          int first, int share) {
  constexpr int NW = 4, D = 512 / TS, HRA = TS, HRB = TS / 2, FA = TS / 32, FB = TS / 64;
  constexpr bool kPaired = EPI == kSwiglu || EPI == kSwigluMx || EPI == kPartialPaired;
  constexpr int kCols = kPaired ? HRB : 2 * HRB;  // output columns
  typedef Half<KA, HRA, NW> HA;
  typedef Half<KB, HRB, NW> HB;

  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t rows = p.m_end - p.m_first;
  const int64_t tm = (rows + HRA - 1) / HRA, tn = (p.N + kCols - 1) / kCols;
  const TileId t = tile_of(id, tm, tn);
  const int64_t m0 = p.m_first + t.m * HRA, n0 = t.n * kCols;
  const int stages = (int)((p.K + (MX ? 255 : 63)) / (MX ? 256 : 64));
  const int count = stages - first < share ? stages - first : share;
  HA a;
  HB b0, b1;
  Lane<KA, HRA, NW> la;
  Lane<KB, HRB, NW> lb;
  la.init(p.lda, wave, lane);
  lb.init(p.ldb, wave, lane);
  const int64_t ka = KA == KC ? (MX ? p.K / 2 : 2 * p.K) : p.K;
  const int64_t kb = KB == KC ? (MX ? p.K / 2 : 2 * p.K) : p.K;
  const int64_t ea = (int64_t)(first + count) * (KA == KC ? kRow : 64);
  const int64_t eb = (int64_t)(first + count) * (KB == KC ? kRow : 64);
  a.init(p.a, m0, p.M, p.lda, ka, ka < ea ? ka : ea);
  b0.init(p.b, n0, p.N, p.ldb, kb, kb < eb ? kb : eb);
  if (kPaired)
    b1.init((const uint8_t*)p.b + p.N * p.ldb, n0, p.N, p.ldb, kb, kb < eb ? kb : eb);
  else
    b1.init(p.b, n0 + HRB, p.N, p.ldb, kb, kb < eb ? kb : eb);
  WaveScales<HRB> scales;  // waves 0 and 1: A's rows; 2 and 3: the halves of B's
  if constexpr (MX) {
    const bool of_a = wave < 2;
    const int64_t all = kPaired ? 2 * (int64_t)p.N : p.N;
    scales.init(of_a ? p.a_scales : p.b_scales, kPaired && wave == 3 ? p.N : 0,
                of_a ? m0 + HRB * wave : kPaired || wave == 2 ? n0 : n0 + HRB, of_a ? p.M : p.N,
                of_a ? p.M : all, p.K, wave * (8 * HRB), true);
  }

  f32x4 acc[2][FA][FB];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) acc[h][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  constexpr int kCopies = HA::kPer + 2 * HB::kPer + (MX ? 1 : 0);  // a stage's, per wave
  auto copy = [&](int s, auto buffer) {
    constexpr int buf = decltype(buffer)::value;
    if constexpr (MX) scales.copy(at.s[buf], s, lane);
    a.copy(at.a[buf], s, wave, la);
    b0.copy(at.b[buf], s, wave, lb);
    b1.copy(at.c[buf], s, wave, lb);
  };
  auto step = [&](int s, auto buffer) {
    constexpr int buf = decltype(buffer)::value;
    wait_vm<(D - 2) * kCopies>();  // stage s has landed; the reads of stage s - 1 are over
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    copy(s + D - 1, std::integral_constant<int, (buf + D - 1) % D>{});
    __builtin_amdgcn_sched_barrier(0);
    Frags<KA, HRA, FA> fa;
    Frags<KB, HRB, FB> fb0, fb1;
    fa.read(at.a[buf], wm * (16 * FA), lane);
    fb0.read(at.b[buf], wn * (16 * FB), lane);
    fb1.read(at.c[buf], wn * (16 * FB), lane);
    u32x2 sm = {};
    uint32_t sn0 = 0, sn1 = 0;
    if constexpr (MX) {
      uint32_t w[2] = {};
      read_scales<FA>(at.s[buf], wm * (16 * FA), lane, w);
      sm = u32x2{w[0], w[1]};
      read_scales<FB>(at.s[buf], HRA + wn * (16 * FB), lane, &sn0);
      read_scales<FB>(at.s[buf], HRA + HRB + wn * (16 * FB), lane, &sn1);
    }
    mma<MX>(acc[0], fb0.v, fa.v, sn0, sm, std::make_integer_sequence<int, 2 * FA * FB>{});
    mma<MX>(acc[1], fb1.v, fa.v, sn1, sm, std::make_integer_sequence<int, 2 * FA * FB>{});
    __builtin_amdgcn_sched_barrier(0);
  };
  each<D - 1>([&](auto i) { copy(first + decltype(i)::value, i); });
  int s = 0;
  for (; s + D <= count; s += D)
    each<D>([&](auto i) { step(first + s + decltype(i)::value, i); });
  each<D - 1>([&](auto i) {
    if (s + decltype(i)::value < count) step(first + s + decltype(i)::value, i);
  });
  wait_vm<0>();  // the copies past the last stage (zeros) land before the LDS is given up
  __builtin_amdgcn_s_barrier();
  const int r = lane & 15, q = lane >> 4;
#pragma unroll
  for (int i = 0; i < FA; ++i) {  // a quarter of the rows an object
    constexpr int kPer = FA / 2;
    const lds_bytes row = (wm ? at.a[2 + i / kPer] : at.a[i / kPer]) + ((i % kPer) * 16 + r) * (4 * TS);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < FB; ++j)
        *(lds_f32x4)(row + (((h * (HRB / 4) + wn * (4 * FB) + j * 4 + q) ^ r) * 16)) = acc[h][i][j];
  }
  wait_lgkm0();
  __builtin_amdgcn_s_barrier();
  store_rows<EPI, TS / 4, TS>(
      p, wave < 2 ? (wave == 0 ? at.a[0] : at.a[1]) : (wave == 2 ? at.a[2] : at.a[3]),
      m0 + wave * (TS / 4), n0, lane);
}
#endif

template <int TS, Kind KA, Kind KB, bool MX, Epilogue EPI>
__global__ __launch_bounds__(256, 1) void tile_kernel(Product p, int share) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (EPI == kPartial || EPI == kPartialPaired)  // blockIdx.y: the share
    p.out = (float*)p.out + ((int64_t)blockIdx.y * (p.m_end - p.m_first) - p.m_first) * p.N *
                                (EPI == kPartialPaired ? 2 : 1);
  Ring<512 / TS> ring;
  if constexpr (TS == 128) {
    FFN_STAGES4(128, MX ? 16 * 128 : 16)
    tile_body<TS, KA, KB, MX, EPI>(p, ring, blockIdx.x, blockIdx.y * share, share);
  } else {
    FFN_STAGES8(64, MX ? 16 * 64 : 16)
    tile_body<TS, KA, KB, MX, EPI>(p, ring, blockIdx.x, blockIdx.y * share, share);
  }
#endif
}

// The backward pass's last three products in one launch: the tiles of each,
// share by share, follow those of the one before. 201 tokens at 1000/680, 232
// work-groups: 11.5 us and 3.9 us for the sums (three launches and a join 31 us);
// the matrix units are busy in 10% of the cycles.
struct Gradients {
  Product product[3];  // dx (NN), dw13, dw2 (TN); aux: the shares' sums, if any
  int first[3];        // their first work-groups
  int tiles[3], share[3];
};
template <int TS>
__device__ __forceinline__ void gradients_body(const Gradients& g, const Ring<512 / TS>& ring) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int group = blockIdx.x;
  const int i = uniform(group < g.first[1] ? 0 : group < g.first[2] ? 1 : 2);
  const int id = uniform((group - g.first[i]) % g.tiles[i]);
  const int share = uniform((group - g.first[i]) / g.tiles[i]);
  Product p = g.product[i];
  if (p.aux) p.aux = (float*)p.aux + share * p.M * p.N;
  if (i == 0)
    tile_body<TS, KC, RC, false, kStoreOrSums>(p, ring, id, share * g.share[i], g.share[i]);
  else
    tile_body<TS, RC, RC, false, kStoreOrSums>(p, ring, id, share * g.share[i], g.share[i]);
#endif
}
template <int TS>
__global__ __launch_bounds__(256, 1) void gradients_kernel(const Gradients g) {
#if defined(__HIP_DEVICE_COMPILE__)
  Ring<512 / TS> ring;
  if constexpr (TS == 128) {
    FFN_STAGES4(128, 16)
    gradients_body<TS>(g, ring);
  } else {
    FFN_STAGES8(64, 16)
    gradients_body<TS>(g, ring);
  }
#endif
}
#undef FFN_STAGE
#undef FFN_STAGES4
#undef FFN_STAGES8

// Adds the shares of K in their order and finishes: one lane (u of the product's)
// four columns of a row; eight lanes a block where h is quantised. Bound by its
// launch and one trip to memory: 3 to 4 us for 333 x 1360 in 4 shares (9 MB).
template <Epilogue EPI>
__device__ __forceinline__ void join_quad(const Product& p, const float* __restrict__ sums,
                                          int shares, int64_t u) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr bool kPaired = EPI == kSwiglu || EPI == kSwigluMx;
  const int64_t quads = p.N / 4;
  const int64_t rows = p.m_end - p.m_first;
  if (u >= rows * quads) return;  // N is a multiple of 32 where lanes work together
  const int64_t row = u / quads, m = p.m_first + row, n = (u - row * quads) * 4;
  const int64_t pitch = (kPaired ? 2 : 1) * (int64_t)p.N;
  const float* src = sums + row * pitch + n;
  f32x4 v = *(const f32x4*)src, up = {};
  if constexpr (kPaired) up = *(const f32x4*)(src + p.N);
  for (int s = 1; s < shares; ++s) {
    src += rows * pitch;
    v += *(const f32x4*)src;
    if constexpr (kPaired) up += *(const f32x4*)(src + p.N);
  }
  if constexpr (EPI == kSwigluMx) {
    emit_mx(p, m, n, v, up, true);
  } else if constexpr (EPI == kSwigluGrad) {
    f32x4 g;
    load_gate_up(p, m, n, g, up);
    emit_grad(p, m, n, v, g, up);
  } else {
    emit<EPI>(p, m, n, v, up);
  }
#endif
}
template <Epilogue EPI>
__global__ __launch_bounds__(256) void join_kernel(const Product p, const float* __restrict__ sums,
                                                   int shares) {
  join_quad<EPI>(p, sums, shares,
                 ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x);
}
__global__ __launch_bounds__(256) void gradients_join_kernel(const Gradients g, const int s0,
                                                             const int s1, const int s2) {
  const int i = (int)blockIdx.x < g.first[1] ? 0 : (int)blockIdx.x < g.first[2] ? 1 : 2;
  join_quad<kStoreBf16>(g.product[i], (const float*)g.product[i].aux, i == 0 ? s0 : i == 1 ? s1 : s2,
                        (int64_t)((int)blockIdx.x - g.first[i]) * 256 + threadIdx.x);
}

// Tile of (AH x 128) x (2 x 128), eight waves (2 x 4), each 64 rows of every A
// half x 32 columns of both B halves. A phase is one A half against both B
// halves, 32 MFMAs (512 cycles) a wave. The two waves of a SIMD run half a
// phase apart: one reads fragments and issues copies while the other's MFMAs
// run, with a barrier after each of the two parts. A half tile is copied into
// its own place as soon as the phase that read it is over.
//
//   AH  buffers  phase  reads      copies                 waits for (at its end)
//   2   2        0      A0 B0 B1   A1 of stage s + 1      A1 of s
//                1      A1         A0 B0 B1 of s + 2      A0 B0 B1 of s + 1
//   1   3        0      A0 B0 B1   all of s + 2           all of s + 1
//
// A part's LDS reads complete before its barrier, so the place is free for the
// copies of the next phase; a copy is waited for before a barrier that every
// wave passes ahead of its reads. Copies have 1.25 (AH = 1: 2) stages to arrive.
//
// Bound by the matrix units at the clock that their power leaves (1.78 to 1.88
// GHz): 4096 x 4096 x 7168 in 160 us, 1.5 PFLOP/s, MFMAs in 85 to 87% of the cycles,
// no LDS bank conflicts. MXFP4 60 us, 4.0 PFLOP/s, MFMAs in 51 to 55% of the cycles
// (7.2 PFLOP/s in registers): a wave waits for copies, LDS or a barrier in 30% of
// its cycles (bf16 21%), its first phase reading all the scales beside the larger
// half of the fragments. Without copies the bf16 product took 0.79 of its time (the
// power goes into the clock), without LDS reads 0.95. Tried
// without gain: four phases of 16 MFMAs (8% slower), the barrier ahead of a
// part's last MFMAs (8% slower), wave priorities, copies among the MFMAs (8%
// slower), fetching ahead into L2 (5% slower), 32 x 32 MFMAs (in registers 1.49
// against 2.03 PFLOP/s), and 256 x 224 tiles where they divide a product into
// whole rounds (the same: CUs without a tile leave the others their power).
// 128 x 256 (AH = 1) takes 0.88 us a stage where 256 x 256 takes 1.42, for sizes
// whose rounds it fills better.
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
  __shared__ __attribute__((aligned(1024))) uint8_t msa0[HA::kBytes], msb0[HB::kBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t msc0[HB::kBytes], msa1[HA::kBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t msb1[HB::kBytes], msc1[HB::kBytes];
  // AH = 2: the second A halves of the two buffers; AH = 1: the third buffer
  __shared__ __attribute__((aligned(1024))) uint8_t msx0[HA::kBytes], msx1[HB::kBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t msx2[AH == 1 ? HB::kBytes : 16];
  constexpr int kScales = MX ? 8 * (AH + 2) * HR : 16;
  __shared__ __attribute__((aligned(16))) uint8_t mss0[kScales], mss1[kScales];
  __shared__ __attribute__((aligned(16))) uint8_t mss2[AH == 1 ? kScales : 16];
  const lds_bytes sa0 = (lds_bytes)msa0, sb0 = (lds_bytes)msb0, sc0 = (lds_bytes)msc0;
  const lds_bytes sa1 = (lds_bytes)msa1, sb1 = (lds_bytes)msb1, sc1 = (lds_bytes)msc1;
  const lds_bytes sx0 = (lds_bytes)msx0, sx1 = (lds_bytes)msx1, sx2 = (lds_bytes)msx2;
  const lds_bytes ss0 = (lds_bytes)mss0, ss1 = (lds_bytes)mss1, ss2 = (lds_bytes)mss2;

  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int64_t tm = (p.m_end - p.m_first + AH * HR - 1) / (AH * HR);
  const int64_t tn = (p.N + kCols - 1) / kCols;
  const TileId t = tile_of(blockIdx.x, tm, tn);
  const int64_t m0 = p.m_first + t.m * (AH * HR), n0 = t.n * kCols;

  HA a0, a1;
  HB b0, b1;
  Lane<KA, HR, NW> la;
  Lane<KB, HR, NW> lb;
  la.init(p.lda, wave, lane);
  lb.init(KA == KC && KB == KC ? p.lda : p.ldb, wave, lane);  // NT: both rows hold K values
  const int64_t ka = KA == KC ? (MX ? p.K / 2 : 2 * p.K) : p.K;
  const int64_t kb = KB == KC ? (MX ? p.K / 2 : 2 * p.K) : p.K;
  a0.init(p.a, m0, p.M, p.lda, ka, ka);
  if constexpr (AH == 2) a1.init(p.a, m0 + HR, p.M, p.lda, ka, ka);
  b0.init(p.b, n0, p.N, p.ldb, kb, kb);
  if (kPaired)
    b1.init((const uint8_t*)p.b + p.N * p.ldb, n0, p.N, p.ldb, kb, kb);
  else
    b1.init(p.b, n0 + HR, p.N, p.ldb, kb, kb);
  const int stages = (int)((p.K + (MX ? 255 : 63)) / (MX ? 256 : 64));

  WaveScales<64> scales;  // two waves a half: A's, then B's
  if constexpr (MX) {
    const int half = wave >> 1, part = (wave & 1) * 64;
    const bool of_a = half < AH;
    const int64_t all = kPaired ? 2 * (int64_t)p.N : p.N;
    scales.init(of_a ? p.a_scales : p.b_scales, kPaired && half == AH + 1 ? p.N : 0,
                (of_a ? m0 + half * HR : kPaired || half == AH ? n0 : n0 + HR) + part,
                of_a ? p.M : p.N, of_a ? p.M : all, p.K, wave * 512, half < AH + 2);
  }
  auto copy_scales = [&](lds_bytes ss, int stage) {
    if constexpr (MX) scales.copy(ss, stage, lane);
  };
  // every wave's copy of scales in flight beside the half tiles' (AH = 1: two waves have none)
  constexpr int kOne = MX && AH == 2 ? 1 : 0;

  f32x4 acc[AH][2][FA][FB];
#pragma unroll
  for (int h = 0; h < 2 * AH; ++h)
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) acc[h / 2][h % 2][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // stages 0 and 1, in the order in which they are waited for
  copy_scales(ss0, 0);
  a0.copy(sa0, 0, wave, la);
  b0.copy(sb0, 0, wave, lb);
  b1.copy(sc0, 0, wave, lb);
  if constexpr (AH == 2) a1.copy(sx0, 0, wave, la);
  copy_scales(ss1, 1);
  a0.copy(sa1, 1, wave, la);
  b0.copy(sb1, 1, wave, lb);
  b1.copy(sc1, 1, wave, lb);
  wait_vm<(AH == 2 ? 4 : 3) * kCopies + kOne>();
  wait_lgkm0();
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  if (wave >= NW / 2) __builtin_amdgcn_s_barrier();  // half a phase behind

  Frags<KA, HR, FA> fa;
  Frags<KB, HR, FB> fb0, fb1;
  u32x2 sm = {}, sm1 = {};
  uint32_t sn0 = 0, sn1 = 0;

#define FFN_MEM_DONE                     \
  wait_lgkm0();                          \
  __builtin_amdgcn_sched_barrier(0);     \
  __builtin_amdgcn_s_barrier();          \
  __builtin_amdgcn_sched_barrier(0);
#define FFN_MMA_DONE                     \
  __builtin_amdgcn_sched_barrier(0);     \
  __builtin_amdgcn_s_barrier();          \
  __builtin_amdgcn_sched_barrier(0);
#define FFN_MMA(ah, sm)                                                                     \
  mma<MX>(acc[ah][0], fb0.v, fa.v, sn0, sm, std::make_integer_sequence<int, 2 * FA * FB>{}); \
  mma<MX>(acc[ah][1], fb1.v, fa.v, sn1, sm, std::make_integer_sequence<int, 2 * FA * FB>{});

  // stage s in buffer `buf`; its scales are read in its first phase, so that their place is
  // free for stage s + 2 in the second
  auto step = [&](int s, auto buffer) {
    constexpr int buf = decltype(buffer)::value;
    constexpr int two = (buf + 2) % 3;  // AH = 1: the buffer of stage s + 2
    const lds_bytes a_now = buf == 0 ? sa0 : buf == 1 ? sa1 : sx0;
    const lds_bytes b0_now = buf == 0 ? sb0 : buf == 1 ? sb1 : sx1;
    const lds_bytes b1_now = buf == 0 ? sc0 : buf == 1 ? sc1 : sx2;
    const lds_bytes ss_now = buf == 0 ? ss0 : buf == 1 ? ss1 : ss2;
    fa.read(a_now, wm * 64, lane);
    fb0.read(b0_now, wn * 32, lane);
    fb1.read(b1_now, wn * 32, lane);
    if constexpr (MX) {
      uint32_t w[2];
      read_scales<FA>(ss_now, wm * 64, lane, w);
      sm = u32x2{w[0], w[1]};
      if constexpr (AH == 2) {
        read_scales<FA>(ss_now, HR + wm * 64, lane, w);
        sm1 = u32x2{w[0], w[1]};
      }
      read_scales<FB>(ss_now, AH * HR + wn * 32, lane, &sn0);
      read_scales<FB>(ss_now, (AH + 1) * HR + wn * 32, lane, &sn1);
    }
    if constexpr (AH == 2) {
      __builtin_amdgcn_sched_barrier(0);  // the reads first: copies wait for their queue
      a1.copy(buf ? sx0 : sx1, s + 1, wave, la);
      wait_vm<4 * kCopies + kOne>();
      FFN_MEM_DONE
      FFN_MMA(0, sm)
      FFN_MMA_DONE
      fa.read(buf ? sx1 : sx0, wm * 64, lane);
      __builtin_amdgcn_sched_barrier(0);
      copy_scales(ss_now, s + 2);
      a0.copy(a_now, s + 2, wave, la);
      b0.copy(b0_now, s + 2, wave, lb);
      b1.copy(b1_now, s + 2, wave, lb);
      wait_vm<4 * kCopies + kOne>();
      FFN_MEM_DONE
      FFN_MMA(1, sm1)
      FFN_MMA_DONE
    } else {
      __builtin_amdgcn_sched_barrier(0);
      copy_scales(two == 0 ? ss0 : two == 1 ? ss1 : ss2, s + 2);
      a0.copy(two == 0 ? sa0 : two == 1 ? sa1 : sx0, s + 2, wave, la);
      b0.copy(two == 0 ? sb0 : two == 1 ? sb1 : sx1, s + 2, wave, lb);
      b1.copy(two == 0 ? sc0 : two == 1 ? sc1 : sx2, s + 2, wave, lb);
      wait_vm<3 * kCopies + kOne>();
      FFN_MEM_DONE
      FFN_MMA(0, sm)
      FFN_MMA_DONE
    }
  };
  int s = 0;
  if constexpr (AH == 2) {
    for (; s + 1 < stages; s += 2) {
      step(s, std::integral_constant<int, 0>{});
      step(s + 1, std::integral_constant<int, 1>{});
    }
    if (s < stages) step(s, std::integral_constant<int, 0>{});
  } else {
    for (; s + 2 < stages; s += 3) {
      step(s, std::integral_constant<int, 0>{});
      step(s + 1, std::integral_constant<int, 1>{});
      step(s + 2, std::integral_constant<int, 2>{});
    }
    if (s < stages) step(s, std::integral_constant<int, 0>{});
    if (s + 1 < stages) step(s + 1, std::integral_constant<int, 1>{});
  }
#undef FFN_MEM_DONE
#undef FFN_MMA_DONE
#undef FFN_MMA
  if (wave < NW / 2) __builtin_amdgcn_s_barrier();
  wait_vm<0>();  // the copies past the last stage (zeros) land before the LDS is given up

  // an A half at a time: 128 rows of 256 columns, 16 an object
  const int r = lane & 15, q = lane >> 4;
  const lds_bytes w0 = wm ? sb1 : sa0;
  const lds_bytes w1 = wm ? sc1 : sb0;
  const lds_bytes w2 = wm ? sx0 : sc0;
  const lds_bytes w3 = wm ? sx1 : sa1;
  const lds_bytes mine = wave < 4 ? (wave < 2 ? (wave == 0 ? sa0 : sb0) : (wave == 2 ? sc0 : sa1))
                                 : (wave < 6 ? (wave == 4 ? sb1 : sc1) : (wave == 6 ? sx0 : sx1));
#pragma unroll
  for (int h = 0; h < AH; ++h) {
    __builtin_amdgcn_s_barrier();  // every wave is done with what the LDS held
#pragma unroll
    for (int i = 0; i < FA; ++i) {
      const lds_bytes row = (i == 0 ? w0 : i == 1 ? w1 : i == 2 ? w2 : w3) + r * 1024;
#pragma unroll
      for (int hb = 0; hb < 2; ++hb)
#pragma unroll
        for (int j = 0; j < FB; ++j)
          *(lds_f32x4)(row + (((hb * 32 + wn * 8 + j * 4 + q) ^ r) * 16)) = acc[h][hb][i][j];
    }
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
    store_rows<EPI, 16, 256>(p, mine, m0 + h * HR + wave * 16, n0, lane);
    wait_lgkm0();
  }
#endif
}

template <Epilogue EPI>
hipError_t join(const Product& p, const void* sums, int shares, hipStream_t stream) {
  const int64_t groups = ((p.m_end - p.m_first) * (p.N / 4) + 255) / 256, y = (groups + (1 << 20) - 1) >> 20;
  hipLaunchKernelGGL((join_kernel<EPI>), dim3((unsigned)((groups + y - 1) / y), (unsigned)y),
                     dim3(256), 0, stream, p, (const float*)sums, shares);
  return hipGetLastError();
}

template <int TS, Layout L, bool MX, Epilogue EPI>
hipError_t launch_small(const Product& p, const Cut& c, dim3 grid, void* split,
                        hipStream_t stream) {
  constexpr Kind KA = L == kTN ? RC : KC, KB = L == kNT ? KC : RC;
  constexpr bool paired = EPI == kSwiglu || EPI == kSwigluMx;
  if (c.shares == 1) {
    hipLaunchKernelGGL((tile_kernel<TS, KA, KB, MX, EPI>), grid, dim3(256), 0, stream, p, c.share);
    return hipGetLastError();
  }
  Product part = p;
  part.out = split;
  hipLaunchKernelGGL((tile_kernel<TS, KA, KB, MX, paired ? kPartialPaired : kPartial>), grid,
                     dim3(256), 0, stream, part, c.share);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : join<EPI>(p, split, c.shares, stream);
}

template <Layout L, bool MX, Epilogue EPI>
hipError_t launch_cut(const Product& p, const Cut& c, void* split, hipStream_t stream) {
  constexpr Kind KA = L == kTN ? RC : KC, KB = L == kNT ? KC : RC;
  const dim3 grid((unsigned)c.groups, c.shares);
  if (c.tile == 2) {
    hipLaunchKernelGGL((big_tile_kernel<2, KA, KB, MX, EPI>), grid, dim3(512), 0, stream, p);
  } else if (c.tile == 1) {
    hipLaunchKernelGGL((big_tile_kernel<1, KA, KB, MX, EPI>), grid, dim3(512), 0, stream, p);
  } else {
    return c.tile == 0 ? launch_small<128, L, MX, EPI>(p, c, grid, split, stream)
                       : launch_small<64, L, MX, EPI>(p, c, grid, split, stream);
  }
  return hipGetLastError();
}

template <Layout L, bool MX, Epilogue EPI>
hipError_t launch(Product p, void* split, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  return each_launch(plan_of(EPI, p.M, p.N, p.K, L, MX), p.M,
                     [&](int64_t first, int64_t end, const Cut& cut) {
                       p.m_first = first;
                       p.m_end = end;
                       return launch_cut<L, MX, EPI>(p, cut, split, stream);
                     });
}

}  // namespace

hipError_t launch_product(Layout layout, Epilogue epilogue, const Product& p, void* split,
                          hipStream_t stream) {
  if (layout == kNT && epilogue == kSwiglu) return launch<kNT, false, kSwiglu>(p, split, stream);
  if (layout == kNT && epilogue == kStoreBf16)
    return launch<kNT, false, kStoreBf16>(p, split, stream);
  if (layout == kNN && epilogue == kSwigluGrad)
    return launch<kNN, false, kSwigluGrad>(p, split, stream);
  if (layout == kNN && epilogue == kStoreBf16)
    return launch<kNN, false, kStoreBf16>(p, split, stream);
  if (layout == kTN && epilogue == kStoreBf16)
    return launch<kTN, false, kStoreBf16>(p, split, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_gradients(const GradientsPlan& plan, const Product (&products)[3], void* split,
                            hipStream_t stream) {
  Gradients g = {};
  int groups = 0;
  for (int i = 0; i < 3; ++i) {
    const Cut& c = plan.cut[i];
    g.product[i] = products[i];
    g.product[i].m_end = products[i].M;
    g.product[i].aux = c.shares > 1 ? (char*)split + plan.sums[i] : nullptr;
    g.first[i] = groups;
    g.tiles[i] = (int)c.groups;
    g.share[i] = c.share;
    groups += (int)c.groups * c.shares;
  }
  if (plan.cut[0].tile == 0)
    hipLaunchKernelGGL(gradients_kernel<128>, dim3(groups), dim3(256), 0, stream, g);
  else
    hipLaunchKernelGGL(gradients_kernel<64>, dim3(groups), dim3(256), 0, stream, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !plan.bytes) return e;
  groups = 0;
  for (int i = 0; i < 3; ++i) {
    g.first[i] = groups;
    if (plan.cut[i].shares > 1)
      groups += (int)((products[i].M * (products[i].N / 4) + 255) / 256);
  }
  hipLaunchKernelGGL(gradients_join_kernel, dim3(groups), dim3(256), 0, stream, g,
                     plan.cut[0].shares, plan.cut[1].shares, plan.cut[2].shares);
  return hipGetLastError();
}

hipError_t launch_product_mx(Epilogue epilogue, const Product& p, void* split,
                             hipStream_t stream) {
  if (epilogue == kStoreBf16) return launch<kNT, true, kStoreBf16>(p, split, stream);
  if (epilogue == kStoreF32) return launch<kNT, true, kStoreF32>(p, split, stream);
  if (epilogue == kSwigluMx) return launch<kNT, true, kSwigluMx>(p, split, stream);
  return hipErrorInvalidValue;
}

}  // namespace ffn
