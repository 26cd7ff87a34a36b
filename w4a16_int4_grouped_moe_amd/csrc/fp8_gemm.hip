// fp8_gemm.hip -- tiled products of FP8 operands with a scale for each block of
// 128 (gfx950).
//
// K advances in stages of 128 bytes of a row, which is one block of scales: the
// stage's products are summed by v_mfma_f32_16x16x128_f8f6f4 from zero, and enter
// the sums by a fused multiply-add with the two scales' product. That MFMA adds
// products eight at a time and cuts each off at a multiple of 2^-13 of the power of two of the
// largest's exponents (measured; the 32-wide FP8 MFMA does the same): up to 2^-10 of
// the sum of magnitudes, 2.6e-5 of a result in the 2-norm on activations with loud
// channels, which is lost in the rounding to bf16 or in the next quantisation. fp32
// results are computed WIDE: the codes widened to bf16, exactly, and summed by
// v_mfma_f32_16x16x32_bf16 in fp32, at half the matrix units' rate. A lane of the
// MFMA holds four consecutive columns n of one row m (its first operand is B), so
// that A's scale is one value a lane and 16 rows, and B's, where its blocks are
// 128 x 128, one scalar.
//
// Operands go from memory into LDS by buffer loads with an LDS destination, in
// whole 128-byte lines; out of range reads zeros (rows past the end, the last
// stage's missing k). Row r holds eight 16-byte pieces, piece c at slot
// c ^ ((r >> 1) & 7): 16 rows at one piece are 16 distinct bank groups of
// ds_read_b128. Lane (r = lane % 16, q = lane / 16) feeds pieces q and 4 + q of
// row r: any order of k within a stage will do that both operands share.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp8_device.h"
#include "fp8_internal.h"

namespace fp8 {
namespace {

// What a lane copies of HR rows x one stage (1 KB a copy, NW waves): rows from `row0` of an
// operand of `rows` rows, or those that `token` names.
template <int HR, int NW>
struct Operand {
  static constexpr int kPer = HR * kRow / 1024 / NW;  // copies per wave
  static_assert(kPer >= 2 && kPer % 2 == 0, "a wave's copies start at an even row group");
  const uint8_t* base;
  int32_t records, end;  // bytes that may be read; bytes of a row
  int piece;             // byte of this lane's piece in even copies (odd ones: ^ 64)
  uint32_t off[kPer];

  __device__ __forceinline__ static int row_of(int wave, int lane, int j) {
    return 8 * (wave * kPer + j) + (lane >> 3);
  }
  __device__ __forceinline__ void init(const uint8_t* ptr, int64_t row0, int64_t rows, int64_t ld,
                                       int64_t K, int wave, int lane) {
    const int64_t left = rows - row0;
    const int valid = left <= 0 ? 0 : left < HR ? (int)left : HR;
    base = ptr + (valid ? row0 * ld : 0);
    records = valid ? (int32_t)((valid - 1) * ld + K) : 0;
    end = (int32_t)K;
    piece = ((lane & 7) ^ (lane >> 4)) * 16;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      off[j] = (uint32_t)(row_of(wave, lane, j) * ld) + (piece ^ ((j & 1) * 64));
  }
  // token(row): the operand's row, or -1; all of the operand fits a resource
  template <typename F>
  __device__ __forceinline__ void gather(const uint8_t* ptr, int64_t rows, int64_t ld, int64_t K,
                                         int wave, int lane, F&& token) {
    base = ptr;
    records = (int32_t)((rows - 1) * ld + K);
    end = (int32_t)K;
    piece = ((lane & 7) ^ (lane >> 4)) * 16;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int32_t t = token(row_of(wave, lane, j));
      off[j] = t < 0 ? kOut : (uint32_t)(t * ld) + (piece ^ ((j & 1) * 64));
    }
  }
  __device__ __forceinline__ void copy(lds_bytes slot, int stage, int wave) const {
    copy(slot, stage, wave, 0, records);
  }
  // the same `shift` bytes further, of `bytes` that may be read
  __device__ __forceinline__ void copy(lds_bytes slot, int stage, int wave, int64_t shift,
                                       int32_t bytes) const {
    const lds_bytes dst = slot + wave * (kPer * 1024);
    const __amdgpu_buffer_rsrc_t res =
        __builtin_amdgcn_make_buffer_rsrc((void*)(base + shift), 0, bytes, kBufferFlags);
    const int k0 = stage * kRow, left = end - k0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool in = (piece ^ ((j & 1) * 64)) < left;
      // kOut + k0 is past every resource too (k0 is below 2^21)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (lds_ptr)(dst + j * 1024), 16,
                                               in ? off[j] + (uint32_t)k0 : kOut, 0, 0, 0);
    }
  }
};

// A wave's copy of scales: 64 rows' of a stage, a lane one, to `at` of the stage's object;
// lanes without a row: zeros
struct WaveScales {
  const float* base;
  int64_t pitch;
  int32_t records, last, at;
  uint32_t off;
  __device__ __forceinline__ void init(const float* scales, int64_t row0, int64_t rows,
                                       int64_t pitch_, int stages, int wave, int lane, bool any) {
    const int64_t left = any ? rows - row0 : 0;
    const int valid = left <= 0 ? 0 : left < 64 ? (int)left : 64;
    base = scales + (valid ? row0 : 0);
    pitch = pitch_;
    records = valid * 4;
    last = stages - 1;
    at = wave * 256;
    off = 4 * lane;
  }
  __device__ __forceinline__ void gather(const float* scales, int64_t rows, int stages, int wave,
                                         int32_t token, bool any) {
    base = scales;
    pitch = rows;
    records = any ? (int32_t)(rows * 4) : 0;
    last = stages - 1;
    at = wave * 256;
    off = token < 0 ? kOut : 4u * token;
  }
  __device__ __forceinline__ void copy(lds_bytes slot, int stage) const {
    const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(base + (stage < last ? stage : last) * pitch), 0, records, kBufferFlags);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (lds_ptr)(slot + at), 4, off, 0, 0, 0);
  }
};

#if defined(__HIP_DEVICE_COMPILE__)
// Four h columns from n of row m, quantised with the 31 lanes that hold the rest of the block
__device__ __forceinline__ void emit_h(const Product& p, int64_t m, int64_t n, const f32x4& g,
                                       const f32x4& u) {
  float h[4];
  uint32_t top = 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    h[r] = g[r] * sigmoid(g[r]) * u[r];
    top = larger(top, magnitude(h[r]));
  }
  top = top_of_16(top);
  top = larger(top, __shfl_xor(top, 16));
  const uint32_t field = scale_field(top);
  const uint32_t c = field == 255 ? 0 : pack4(h, scale_inverse(field));
  if (m >= p.M || n >= p.N) return;
  *(uint32_t*)((uint8_t*)p.out + m * p.N + n) = c;
  if ((n & 127) == 0) p.aux[n / kBlock * p.M + m] = scale_value(field);
}

// ROWS rows from m0, 4 x COLS bytes each in LDS (16-byte piece c of row r at c ^ (r % 16)): a
// lane four columns of one (kSwiglu: of its gate and its up columns)
template <Epilogue EPI, int ROWS, int COLS>
__device__ __forceinline__ void store_rows(const Product& p, lds_bytes lds, int64_t m0, int64_t n0,
                                           int lane) {
  constexpr bool kPaired = EPI == kSwiglu;
  constexpr int kLanes = COLS / (kPaired ? 8 : 4);  // a row's lanes
  constexpr int kRowsAtOnce = 64 / kLanes, kTurns = ROWS / kRowsAtOnce;
  constexpr int kMost = kPaired ? 4 : 8, kBatch = kTurns < kMost ? kTurns : kMost;
  const int c = lane % kLanes;
  const int64_t n = n0 + 4 * c, N = p.N;
#pragma unroll
  for (int t = 0; t < kTurns; t += kBatch) {
    f32x4 v[kBatch], up[kBatch];
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
      if constexpr (EPI == kSwiglu) {
        emit_h(p, m, n, v[k], up[k]);
      } else {
        if (m >= p.M || n >= N) continue;
        if constexpr (EPI == kStoreBf16) {
          *(u32x2*)((uint16_t*)p.out + m * N + n) =
              u32x2{pack2(v[k][0], v[k][1]), pack2(v[k][2], v[k][3])};
        } else {
          *(f32x4*)((float*)p.out + m * N + n) = v[k];
        }
      }
    }
  }
}
#endif

// An object a half tile and a stage's scales: the compiler then sees which copies a read has to
// wait for. x: AH = 2: the second A halves of the two buffers; AH = 1: the third buffer.
struct BigLds {
  lds_bytes a0, b0, c0, a1, b1, c1, x0, x1, x2, s0, s1, s2;
};
#define FP8_BIG_LDS(third)                                                                  \
  __shared__ __attribute__((aligned(1024))) uint8_t msa0[kHalf], msb0[kHalf], msc0[kHalf];  \
  __shared__ __attribute__((aligned(1024))) uint8_t msa1[kHalf], msb1[kHalf], msc1[kHalf];  \
  __shared__ __attribute__((aligned(1024))) uint8_t msx0[kHalf], msx1[kHalf];               \
  __shared__ __attribute__((aligned(1024))) uint8_t msx2[(third) ? kHalf : 16];             \
  __shared__ __attribute__((aligned(16))) uint8_t mss0[2048], mss1[2048];                   \
  __shared__ __attribute__((aligned(16))) uint8_t mss2[(third) ? 2048 : 16];                \
  const BigLds lds = {(lds_bytes)msa0, (lds_bytes)msb0, (lds_bytes)msc0, (lds_bytes)msa1,   \
                      (lds_bytes)msb1, (lds_bytes)msc1, (lds_bytes)msx0, (lds_bytes)msx1,   \
                      (lds_bytes)msx2, (lds_bytes)mss0, (lds_bytes)mss1, (lds_bytes)mss2};
constexpr int kHalf = 128 * kRow;

#if defined(__HIP_DEVICE_COMPILE__)
// Tile of (AH x 128) x (2 x 128), eight waves (2 x 4), each 64 rows of every A
// half x 32 columns of both B halves (kSwiglu: gate and up). A phase is one A half
// against both B halves, 16 MFMAs a wave of 32 cycles each. The two waves of a SIMD run half a phase
// apart: one reads fragments and issues copies while the other's MFMAs and
// multiply-adds run, with a barrier after each of the two parts. A half tile is
// copied into its own place as soon as the phase that read it is over.
//
//   AH  buffers  phase  reads      copies                 waits for (at its end)
//   2   2        0      A0 B0 B1   A1 of stage s + 1      A1 of s
//                1      A1         A0 B0 B1 of s + 2      A0 B0 B1 of s + 1
//   1   3        0      A0 B0 B1   all of s + 2           all of s + 1
//
// The scales travel with A0: they are read in the first phase. Beside each MFMA of 32 cycles
// go the four multiply-adds of an earlier one.
//
// Bound by the matrix units at the clock that their power leaves (1.76 to 2.0 GHz), and by what
// goes around them: 4096 x 4096 x 7168 in 101 us, 2.4 PFLOP/s (a library product with a single
// scale 84 us), MFMAs in 67% of the cycles, a wave waiting in 27% of its own, no LDS conflicts.
// fp32 results (128 x 256 alone, and twice the MFMA cycles for widened operands) 4096 x 7168 x 4096
// in 251 to 275 us, 0.9 PFLOP/s, MFMAs in 52% of the cycles, and 3.5 rounds of tiles in four.
//
// idle: this wave's rows are all padding. kPairs: `tiles` column tiles one after the other, the
// copies of the next under way while one is stored, straight from the registers to the pairs'
// rows (`rows`: the pairs of the block's rows).
template <int AH, Mode MODE, Epilogue EPI, bool WIDE>
__device__ __forceinline__ void big_tile(Product p, const BigLds& lds, int64_t m0, int64_t n0,
                                         bool idle, int tiles, lds_i32 rows) {
  constexpr bool kSpan = EPI == kPairs;
  constexpr int NW = 8, HR = 128, FA = 4, FB = 2;
  constexpr bool kPaired = EPI == kSwiglu, kRows = MODE == kRowScales;
  typedef Operand<HR, NW> Half;
  constexpr int kCopies = Half::kPer;
  const lds_bytes sa0 = lds.a0, sb0 = lds.b0, sc0 = lds.c0, sa1 = lds.a1, sb1 = lds.b1;
  const lds_bytes sc1 = lds.c1, sx0 = lds.x0, sx1 = lds.x1, sx2 = lds.x2;
  const lds_bytes ss0 = lds.s0, ss1 = lds.s1, ss2 = lds.s2;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int stages = (int)((p.K + kRow - 1) / kRow);

  Half a[AH], b0, b1;
  WaveScales scales;  // waves 0 .. 2 AH - 1: A's rows; kRows: 4 .. 7: B's
  if constexpr (MODE == kTokens) {
    const int64_t tokens = p.a_rows;
    auto token = [&](int row) {
      const int32_t pair = p.sorted[m0 + row];
      return (uint32_t)pair < (uint32_t)p.pairs ? pair / p.top_k : -1;
    };
#pragma unroll
    for (int h = 0; h < AH; ++h)
      a[h].gather(p.a, tokens, p.lda, p.K, wave, lane, [&](int row) { return token(h * HR + row); });
    scales.gather(p.a_scales, tokens, stages, wave, wave < 2 * AH ? token(wave * 64 + lane) : -1,
                  wave < 2 * AH);
  } else {
#pragma unroll
    for (int h = 0; h < AH; ++h) a[h].init(p.a, m0 + h * HR, p.M, p.lda, p.K, wave, lane);
    const bool of_b = kRows && wave >= 4;
    scales.init(of_b ? p.b_scales : p.a_scales, of_b ? n0 + (wave - 4) * 64 : m0 + wave * 64,
                of_b ? p.N : p.M, of_b ? p.sb_stage : p.a_rows, stages, wave, lane,
                of_b || wave < 2 * AH);
  }
  b0.init(p.b, n0, p.N, p.ldb, p.K, wave, lane);
  if (kPaired)
    b1.init(p.b + p.N * p.ldb, n0, p.N, p.ldb, p.K, wave, lane);
  else
    b1.init(p.b, n0 + HR, p.N, p.ldb, p.K, wave, lane);
  // B's square scales of the halves; a half without columns takes the other's
  // (constant address space: scalar loads, which do not count among the copies)
  const const_f32 sq0 = (const_f32)(p.b_scales + n0 / kBlock * p.sb_row);
  const const_f32 sq1 = kPaired ? sq0 + p.N / kBlock * p.sb_row : n0 + HR < p.N ? sq0 + p.sb_row : sq0;

  f32x4 acc[AH][2][FA][FB];
#pragma unroll
  for (int h = 0; h < 2 * AH; ++h)
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) acc[h / 2][h % 2][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // stage s of tile c; `ahead` stages further: its stage and tile (kSpan; past the last tile a
  // stage past K, whose copies are zeros)
  int s = 0, c = 0;
  struct At {
    int stage, tile;
  };
  const auto ahead = [&](int by) {
    At t{s + by, c};
    if constexpr (kSpan) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (t.stage >= stages) t.stage -= stages, ++t.tile;
      if (t.tile >= tiles) t = At{stages, c};
    }
    return t;
  };
  const auto copy_b = [&](lds_bytes slot0, lds_bytes slot1, const At& t) {
    if constexpr (kSpan) {
      const int64_t shift = t.tile * 256 * p.ldb;
      const int32_t whole = (int32_t)((HR - 1) * p.ldb + p.K);
      b0.copy(slot0, t.stage, wave, shift, whole);
      b1.copy(slot1, t.stage, wave, shift, n0 + t.tile * 256 + HR < p.N ? whole : 0);
    } else {
      b0.copy(slot0, t.stage, wave);
      b1.copy(slot1, t.stage, wave);
    }
  };
  // stages 0 and 1, in the order in which they are waited for
  scales.copy(ss0, 0);
  a[0].copy(sa0, 0, wave);
  copy_b(sb0, sc0, At{0, 0});
  if constexpr (AH == 2) a[1].copy(sx0, 0, wave);
  const At second = ahead(1);
  scales.copy(ss1, second.stage);
  a[0].copy(sa1, second.stage, wave);
  copy_b(sb1, sc1, second);
  wait_vm<(AH == 2 ? 4 : 3) * kCopies + 1>();
  wait_lgkm0();
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  if (wave >= NW / 2) __builtin_amdgcn_s_barrier();  // half a phase behind

  Frags<FA> fa;
  Frags<FB> fb[2];
  Wide<FB> wide[2];
  float sa[AH][FA];
  ColumnScales<kRows, FB> cs[2];

#define FP8_MEM_DONE                     \
  wait_lgkm0();                          \
  __builtin_amdgcn_sched_barrier(0);     \
  __builtin_amdgcn_s_barrier();          \
  __builtin_amdgcn_sched_barrier(0);
#define FP8_MMA_DONE                     \
  __builtin_amdgcn_sched_barrier(0);     \
  __builtin_amdgcn_s_barrier();          \
  __builtin_amdgcn_sched_barrier(0);
#define FP8_MMA(ah)                                              \
  if (!idle) {                                                   \
    if constexpr (WIDE)                                          \
      mma_wide<kRows, 2, FA, FB>(acc[ah], wide, fa, sa[ah], cs); \
    else                                                         \
      mma<kRows, 2, FA, FB>(acc[ah], fb, fa, sa[ah], cs);        \
    hold(acc[ah]);                                               \
  }

  // B's square scales of the next stage, asked for ahead of a phase's MFMAs: its scalar loads
  // (each stage's from another line) would hold up the wait for the fragments
  float sq_next0 = 0.f, sq_next1 = 0.f;
  const auto ask = [&](const At& t) {
    if constexpr (!kRows) {
      int64_t at = (t.stage < stages ? t.stage : stages - 1) * p.sb_stage;
      if constexpr (kSpan) at += 2 * t.tile * p.sb_row;
      sq_next0 = sq0[at];
      if constexpr (kSpan)
        sq_next1 = sq0[n0 + t.tile * 256 + HR < p.N ? at + p.sb_row : at];
      else
        sq_next1 = sq1[at];
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  ask(At{0, 0});
  const auto store_pairs = [&] {
    const int64_t n = n0 + c * 256 + wn * 32 + 4 * (lane >> 4);
#pragma unroll
    for (int h = 0; h < AH; ++h)
#pragma unroll
      for (int i = 0; i < FA; ++i) {
        const int32_t pair = rows[h * HR + wm * 64 + i * 16 + (lane & 15)];
        float* const out = (float*)p.out + (int64_t)pair * p.N + n;
        if ((uint32_t)pair < (uint32_t)p.pairs) {
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            if (hb == 1 && n0 + c * 256 + HR >= p.N) continue;
#pragma unroll
            for (int j = 0; j < FB; ++j) *(f32x4*)(out + hb * HR + j * 16) = acc[h][hb][i][j];
          }
        }
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
          for (int j = 0; j < FB; ++j) acc[h][hb][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
  };
  // stage s in buffer `buf`; its scales are read in its first phase, so that their place is
  // free for stage s + 2 in the second
  auto step = [&](auto buffer) {
    constexpr int buf = decltype(buffer)::value;
    constexpr int two = (buf + 2) % 3;  // AH = 1: the buffer of stage s + 2
    const lds_bytes a_now = buf == 0 ? sa0 : buf == 1 ? sa1 : sx0;
    const lds_bytes b0_now = buf == 0 ? sb0 : buf == 1 ? sb1 : sx1;
    const lds_bytes b1_now = buf == 0 ? sc0 : buf == 1 ? sc1 : sx2;
    const lds_bytes ss_now = buf == 0 ? ss0 : buf == 1 ? ss1 : ss2;
    const At one_on = ahead(1), two_on = ahead(2);
    if constexpr (!kRows) cs[0].set(sq_next0), cs[1].set(sq_next1);
    if (!idle) {
      fa.read(a_now, wm * 64, lane);
      fb[0].read(b0_now, wn * 32, lane);
      fb[1].read(b1_now, wn * 32, lane);
#pragma unroll
      for (int h = 0; h < AH; ++h)
#pragma unroll
        for (int i = 0; i < FA; ++i)
          sa[h][i] = *(lds_f32)(ss_now + (h * HR + wm * 64 + i * 16 + (lane & 15)) * 4);
      cs[0].read(ss_now + 1024, wn * 32, lane);
      cs[1].read(ss_now + 1024, HR + wn * 32, lane);
    }
    if constexpr (AH == 2) {
      __builtin_amdgcn_sched_barrier(0);  // the reads first: copies wait for their queue
      a[1].copy(buf ? sx0 : sx1, one_on.stage, wave);
      wait_vm<4 * kCopies + 1>();
      FP8_MEM_DONE
      FP8_MMA(0)
      FP8_MMA_DONE
      fa.read(buf ? sx1 : sx0, wm * 64, lane);
      __builtin_amdgcn_sched_barrier(0);
      scales.copy(ss_now, two_on.stage);
      a[0].copy(a_now, two_on.stage, wave);
      copy_b(b0_now, b1_now, two_on);
      wait_vm<4 * kCopies + 1>();
      FP8_MEM_DONE
      ask(one_on);
      FP8_MMA(AH - 1)
    } else {
      __builtin_amdgcn_sched_barrier(0);
      scales.copy(two == 0 ? ss0 : two == 1 ? ss1 : ss2, two_on.stage);
      a[0].copy(two == 0 ? sa0 : two == 1 ? sa1 : sx0, two_on.stage, wave);
      copy_b(two == 0 ? sb0 : two == 1 ? sb1 : sx1, two == 0 ? sc0 : two == 1 ? sc1 : sx2, two_on);
      if constexpr (WIDE) wide[0].set(fb[0]), wide[1].set(fb[1]);
      wait_vm<3 * kCopies + 1>();
      FP8_MEM_DONE
      ask(one_on);
      FP8_MMA(0)
    }
    ++s;
    if constexpr (kSpan)
      if (s == stages) {  // the tile's end; what it stores is waited for with the copies after it
        store_pairs();
        s = 0;
        ++c;
      }
    FP8_MMA_DONE
  };
  const int all = kSpan ? stages * tiles : stages;
  int n = 0;
  if constexpr (AH == 2) {
    for (; n + 1 < all; n += 2) {
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
    }
    if (n < all) step(std::integral_constant<int, 0>{});
  } else {
    for (; n + 2 < all; n += 3) {
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{});
    }
    if (n < all) step(std::integral_constant<int, 0>{});
    if (n + 1 < all) step(std::integral_constant<int, 1>{});
  }
#undef FP8_MEM_DONE
#undef FP8_MMA_DONE
#undef FP8_MMA
  if (wave < NW / 2) __builtin_amdgcn_s_barrier();
  wait_vm<0>();  // the copies past the last stage (zeros) land before the LDS is given up
  if constexpr (kSpan) return;

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
}
#endif

template <int AH, Mode MODE, Epilogue EPI, bool WIDE>
__global__ __launch_bounds__(512, 2) void big_tile_kernel(const Product p) {
#if defined(__HIP_DEVICE_COMPILE__)
  FP8_BIG_LDS(AH == 1)
  const int64_t tm = (p.m_end - p.m_first + AH * 128 - 1) / (AH * 128), tn = (p.N + 255) / 256;
  const TileId t = tile_of(blockIdx.x, tm, tn);
  big_tile<AH, MODE, EPI, WIDE>(p, lds, p.m_first + t.m * (AH * 128), t.n * 256, false, 1, {});
#endif
}

// The experts' products, a work-group a bucket block of 256 rows x 256 columns (kSwiglu: 128
// gate, 128 up; kPairs: several such in turn): a block of 128 pairs or fewer as a 128 x 256 tile,
// of 64 or fewer on half the waves, which leaves the time to the weights' copies. 2048 tokens
// over 48 of 384 experts at 7168/2048 (43 rows each): 1.41 GB in 279 us, 5.0 TB/s, and 0.70 GB in
// 168 us, 4.2 TB/s. 4096 tokens over 48 experts (683 rows each, 768 with padding): 900 to 1030 us,
// 2.1 to 2.4 PFLOP/s on what the tiles compute, at 1.76 GHz; the second product 650 to 705 us,
// of which its 16 stages a tile are 60%: each round of tiles writes 67 MB of y at once.
template <Mode MODE, Epilogue EPI>
__global__ __launch_bounds__(512, 2) void experts_kernel(Product p) {
#if defined(__HIP_DEVICE_COMPILE__)
  FP8_BIG_LDS(true)
  __shared__ int32_t rows[EPI == kPairs ? kBigRows : 1];
  constexpr int kCols = EPI == kSwiglu ? 128 : 256;
  const int64_t tm = *p.n_padded / kBigRows, tn = (p.N + kCols - 1) / kCols;
  const int span = EPI == kPairs ? experts_span(tm, tn) : 1;
  const int64_t across = (tn + span - 1) / span;
  if ((int64_t)blockIdx.x >= tm * across) return;  // the grid is sized for the most buckets
  const TileId t = tile_of(blockIdx.x, tm, across);
  const int64_t m0 = t.m * kBigRows, n0 = t.n * span * kCols;
  const int tiles = (int)(tn - t.n * span < span ? tn - t.n * span : span);
  const int64_t b_rows = EPI == kSwiglu ? 2 * (int64_t)p.N : p.N;
  const int64_t e = uniform(p.block_expert[t.m]);
  p.b += e * b_rows * p.ldb;
  p.b_scales += e * (b_rows / kBlock) * p.sb_row;
  if constexpr (EPI == kPairs)  // (the first barrier comes before its first use)
    if (threadIdx.x < kBigRows) rows[threadIdx.x] = p.sorted[m0 + threadIdx.x];
  // a block's pairs come first
  const auto filled = [&](int row) {
    return uniform((uint32_t)p.sorted[m0 + row] < (uint32_t)p.pairs) != 0;
  };
  if (filled(128)) {
    big_tile<2, MODE, EPI, false>(p, lds, m0, n0, false, tiles, (lds_i32)rows);
  } else {
    const bool idle = (threadIdx.x >> 8) != 0 && !filled(64);
    big_tile<1, MODE, EPI, false>(p, lds, m0, n0, uniform(idle) != 0, tiles, (lds_i32)rows);
  }
#endif
}
#undef FP8_BIG_LDS

// A small tile's ring of stages (four of 128 x 128, eight of 64 x 64): an object
// a stage and operand, so that the compiler sees which copies a read has to wait
// for. `a` also holds the tile on its way out.
template <int D>
struct Ring {
  lds_bytes a[D], b[D], s[D];
};
#define FP8_STAGE(i, tile)                                               \
  __shared__ __attribute__((aligned(1024))) uint8_t sa##i[(tile) * kRow]; \
  __shared__ __attribute__((aligned(1024))) uint8_t sb##i[(tile) * kRow]; \
  __shared__ __attribute__((aligned(16))) uint8_t ss##i[1024];            \
  ring.a[i] = (lds_bytes)sa##i, ring.b[i] = (lds_bytes)sb##i, ring.s[i] = (lds_bytes)ss##i;
#define FP8_STAGES4(tile) \
  FP8_STAGE(0, tile) FP8_STAGE(1, tile) FP8_STAGE(2, tile) FP8_STAGE(3, tile)
#define FP8_STAGES8(tile) \
  FP8_STAGES4(tile) FP8_STAGE(4, tile) FP8_STAGE(5, tile) FP8_STAGE(6, tile) FP8_STAGE(7, tile)

#if defined(__HIP_DEVICE_COMPILE__)
// Tile of TS x TS, TS = 128 or 64: four waves (2 x 2), for launches that leave CUs idle: a ring
// of D stages, copied D - 1 ahead, and one barrier a stage. The stages from `first`, at most
// `share` of them. 64 x 64 takes 0.32 us a stage (0.49 with fp32 results), 128 x 128 0.78 (1.20)
// for four times the work, and 5 to 7 us besides. Neither memory nor the matrix units bound it:
// 777 x 1000 x 1008 (9.3 us) keeps the matrix units busy in 10% of the cycles, a wave issues in
// 42% of its own and waits for copies, LDS and the barrier in 39%.
template <int TS, Mode MODE, Epilogue EPI, bool WIDE>
__device__ __forceinline__ void tile_body(const Product& p, const Ring<512 / TS>& at, int64_t id,
                                          int first, int share) {
  constexpr int NW = 4, D = 512 / TS, F = TS / 32;
  constexpr bool kRows = MODE == kRowScales;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t tm = (p.m_end - p.m_first + TS - 1) / TS, tn = (p.N + TS - 1) / TS;
  const TileId t = tile_of(id, tm, tn);
  const int64_t m0 = p.m_first + t.m * TS, n0 = t.n * TS;
  const int stages = (int)((p.K + kRow - 1) / kRow);
  const int count = stages - first < share ? stages - first : share;
  const int64_t end = (int64_t)(first + count) * kRow, K = p.K < end ? p.K : end;
  Operand<TS, NW> a, b;
  a.init(p.a, m0, p.M, p.lda, K, wave, lane);
  b.init(p.b, n0, p.N, p.ldb, K, wave, lane);
  WaveScales scales;  // waves 0 and 1: A's rows, kRows: 2 and 3: B's
  const bool of_b = wave >= 2;
  scales.init(of_b ? p.b_scales : p.a_scales, (of_b ? n0 : m0) + (wave & 1) * 64,
              of_b ? p.N : p.M, of_b ? p.sb_stage : p.a_rows, stages, wave, lane,
              (wave & 1) * 64 < TS && (kRows || !of_b));
  const const_f32 sq = (const_f32)(p.b_scales + n0 / kBlock * p.sb_row);

  f32x4 acc[1][F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[0][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  float sq_next = kRows ? 0.f : sq[first * p.sb_stage];
  constexpr int kCopies = 2 * Operand<TS, NW>::kPer + 1;  // a stage's, per wave
  auto copy = [&](int s, auto buffer) {
    constexpr int buf = decltype(buffer)::value;
    scales.copy(at.s[buf], s);
    a.copy(at.a[buf], s, wave);
    b.copy(at.b[buf], s, wave);
  };
  auto step = [&](int s, auto buffer) {
    constexpr int buf = decltype(buffer)::value;
    ColumnScales<kRows, F> cs[1];
    if constexpr (!kRows) cs[0].set(sq_next);
    wait_vm<(D - 2) * kCopies>();  // stage s has landed; the reads of stage s - 1 are over
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    copy(s + D - 1, std::integral_constant<int, (buf + D - 1) % D>{});
    if constexpr (!kRows)  // the next stage's, on its way during this one
      sq_next = sq[(s + 1 < stages ? s + 1 : s) * p.sb_stage];
    __builtin_amdgcn_sched_barrier(0);
    Frags<F> fa, fb[1];
    float sa[F];
    fa.read(at.a[buf], wm * (16 * F), lane);
    fb[0].read(at.b[buf], wn * (16 * F), lane);
#pragma unroll
    for (int i = 0; i < F; ++i)
      sa[i] = *(lds_f32)(at.s[buf] + ((wm * F + i) * 16 + (lane & 15)) * 4);
    cs[0].read(at.s[buf] + 512, wn * (16 * F), lane);
    if constexpr (WIDE) {
      Wide<F> wide[1];
      wide[0].set(fb[0]);
      mma_wide<kRows, 1, F, F>(acc, wide, fa, sa, cs);
    } else {
      mma<kRows, 1, F, F>(acc, fb, fa, sa, cs);
    }
    hold(acc);
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
  for (int i = 0; i < F; ++i) {  // a quarter of the rows an object
    constexpr int kPer = F / 2;
    const lds_bytes row =
        (wm ? at.a[2 + i / kPer] : at.a[i / kPer]) + ((i % kPer) * 16 + r) * (4 * TS);
#pragma unroll
    for (int j = 0; j < F; ++j)
      *(lds_f32x4)(row + (((wn * (4 * F) + j * 4 + q) ^ r) * 16)) = acc[0][i][j];
  }
  wait_lgkm0();
  __builtin_amdgcn_s_barrier();
  store_rows<EPI, TS / 4, TS>(
      p, wave < 2 ? (wave == 0 ? at.a[0] : at.a[1]) : (wave == 2 ? at.a[2] : at.a[3]),
      m0 + wave * (TS / 4), n0, lane);
}
#endif

template <int TS, Mode MODE, Epilogue EPI, bool WIDE>
__global__ __launch_bounds__(256, 1) void tile_kernel(Product p, int share) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (EPI == kPartial)  // blockIdx.y: the share
    p.out = (float*)p.out + ((int64_t)blockIdx.y * (p.m_end - p.m_first) - p.m_first) * p.N;
  Ring<512 / TS> ring;
  if constexpr (TS == 128) {
    FP8_STAGES4(128)
    tile_body<TS, MODE, EPI, WIDE>(p, ring, blockIdx.x, blockIdx.y * share, share);
  } else {
    FP8_STAGES8(64)
    tile_body<TS, MODE, EPI, WIDE>(p, ring, blockIdx.x, blockIdx.y * share, share);
  }
#endif
}
#undef FP8_STAGE
#undef FP8_STAGES4
#undef FP8_STAGES8

// Adds the shares of K in their order: a lane four columns of a row
template <Epilogue EPI>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ sums, int shares,
                                                   int64_t quads, void* __restrict__ out) {
  const int64_t u = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  if (u >= quads) return;
  f32x4 v = ((const f32x4*)sums)[u];
  for (int s = 1; s < shares; ++s) v += ((const f32x4*)sums)[s * quads + u];
  if constexpr (EPI == kStoreBf16)
    ((u32x2*)out)[u] = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
  else
    ((f32x4*)out)[u] = v;
}

// rows [p.m_first, p.m_end), as are launch_small's
template <int AH, Mode MODE, Epilogue EPI, bool WIDE = false>
hipError_t launch_big(Product p, hipStream_t stream) {
  const int64_t tn = (p.N + 255) / 256, end = p.m_end;
  const int64_t most = kMaxGroups / tn * (AH * 128);
  for (int64_t m = p.m_first; m < end; m += most) {
    p.m_first = m;
    p.m_end = end - m < most ? end : m + most;
    const int64_t tm = (p.m_end - m + AH * 128 - 1) / (AH * 128);
    hipLaunchKernelGGL((big_tile_kernel<AH, MODE, EPI, WIDE>), dim3((unsigned)(tm * tn)),
                       dim3(512), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int TS, Mode MODE, Epilogue EPI>
hipError_t launch_small(Product p, const Cut& c, void* split, hipStream_t stream) {
  constexpr bool kWide = EPI == kStoreF32;
  const dim3 grid((unsigned)c.groups, c.shares);
  if (c.shares == 1) {
    hipLaunchKernelGGL((tile_kernel<TS, MODE, EPI, kWide>), grid, dim3(256), 0, stream, p, c.share);
    return hipGetLastError();
  }
  void* const out = (char*)p.out + p.m_first * p.N * (EPI == kStoreF32 ? 4 : 2);
  p.out = split;
  hipLaunchKernelGGL((tile_kernel<TS, MODE, kPartial, kWide>), grid, dim3(256), 0, stream, p,
                     c.share);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t quads = (p.m_end - p.m_first) * (p.N / 4), groups = (quads + 255) / 256;
  const int64_t y = (groups + (1 << 20) - 1) >> 20;
  hipLaunchKernelGGL(join_kernel<EPI>, dim3((unsigned)((groups + y - 1) / y), (unsigned)y),
                     dim3(256), 0, stream, (const float*)split, c.shares, quads, out);
  return hipGetLastError();
}

template <Mode MODE, Epilogue EPI>
hipError_t launch_cut(const Product& p, const Cut& c, void* split, hipStream_t stream) {
  if constexpr (EPI == kStoreBf16)
    if (c.tile == 2) return launch_big<2, MODE, EPI>(p, stream);
  if (c.tile == 1) return launch_big<1, MODE, EPI, EPI == kStoreF32>(p, stream);
  return c.tile == 0 ? launch_small<128, MODE, EPI>(p, c, split, stream)
                     : launch_small<64, MODE, EPI>(p, c, split, stream);
}

template <Mode MODE, Epilogue EPI>
hipError_t launch(Product p, void* split, hipStream_t stream) {
  const Plan plan = plan_of(EPI == kStoreF32, MODE == kRowScales, p.M, p.N, p.K);
  p.m_end = plan.first ? plan.first : p.M;
  const hipError_t e = launch_cut<MODE, EPI>(p, plan.whole, split, stream);
  if (e != hipSuccess || !plan.first) return e;
  p.m_first = plan.first;
  p.m_end = p.M;
  return launch_cut<MODE, EPI>(p, plan.rest, split, stream);
}

}  // namespace

hipError_t launch_product(Mode mode, Epilogue epilogue, const Product& p, void* split,
                          hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  if (mode == kSquare && epilogue == kStoreBf16) return launch<kSquare, kStoreBf16>(p, split, stream);
  if (mode == kSquare && epilogue == kStoreF32) return launch<kSquare, kStoreF32>(p, split, stream);
  if (mode == kRowScales && epilogue == kStoreBf16)
    return launch<kRowScales, kStoreBf16>(p, split, stream);
  if (mode == kRowScales && epilogue == kStoreF32)
    return launch<kRowScales, kStoreF32>(p, split, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_experts(Epilogue epilogue, const Product& p, hipStream_t stream) {
  const int64_t cols = epilogue == kSwiglu ? 128 : 256;
  const dim3 grid((unsigned)(p.M / kBigRows * ((p.N + cols - 1) / cols)));
  if (epilogue == kSwiglu)
    hipLaunchKernelGGL((experts_kernel<kTokens, kSwiglu>), grid, dim3(512), 0, stream, p);
  else if (epilogue == kPairs)
    hipLaunchKernelGGL((experts_kernel<kBuckets, kPairs>), grid, dim3(512), 0, stream, p);
  else
    return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace fp8
