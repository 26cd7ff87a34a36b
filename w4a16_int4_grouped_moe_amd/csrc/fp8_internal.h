// fp8_internal.h -- what the FP8 block operators' host code and kernels share.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8 {

constexpr int kBlock = 128;  // values of a row under one scale; bytes of a stage of K
__host__ __device__ inline int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// x [rows, width] (type: MOE_TYPE_*) -> codes [rows, width], scales (see moe_fp8.h)
hipError_t launch_quantize(const void* x, int32_t type, int64_t rows, int32_t width, int32_t block,
                           uint8_t* codes, float* scales, hipStream_t stream);
hipError_t launch_clear(void* out, int64_t bytes, hipStream_t stream);  // a multiple of 16
hipError_t launch_dequantize(const uint8_t* codes, const float* scales, int64_t rows,
                             int32_t width, int32_t block, int32_t type, void* out,
                             hipStream_t stream);
// What the gradients' products read: B's codes [cols, width] transposed (b_t), dout bf16 [rows,
// cols] in 1 x 128 blocks (dout_codes) and its transpose in such blocks (dout_t), and a's
// transpose (a bf16 [rows, width]). Rows of codes are 128 blocks_of(their width) bytes, zeros
// behind the values; scales as moe_fp8.h has them. What is NULL is not computed (dout_codes or
// dout_t is given).
struct Prepare {
  const void* dout;
  const void* a;
  const uint8_t* b;
  int64_t rows;
  int32_t cols, width;
  uint8_t* b_t;
  uint8_t* dout_codes;
  float* dout_scales;
  uint8_t* dout_t;
  float* dout_t_scales;
  uint8_t* a_t;
  float* a_t_scales;
};
hipError_t launch_prepare(const Prepare& p, hipStream_t stream);

// D[m, n] = sum over the stages (128 bytes of a row) of sa(m, stage) sb(n, stage) times the
// stage's sum of A(m, k) B(n, k).
constexpr int64_t kMaxGroups = 0x7fffff;  // of 512 lanes in a launch of fewer than 2^32
enum Mode {
  kSquare = 0,   // B's scales: 128 x 128 blocks
  kRowScales = 1,  // B's scales: 1 x 128 blocks
  kTokens = 2,   // experts, square scales: A's rows are the tokens of bucketed pairs
  kBuckets = 3,  // experts, square scales: A's rows are bucket rows
};
enum Epilogue {
  kStoreBf16 = 0,
  kStoreF32 = 1,
  kSwiglu = 2,   // kTokens: B's rows [0, N) gate, [N, 2N) up; out codes of h, aux its scales
  kPairs = 3,    // kBuckets: out fp32, a bucket row's at its pair's row
  kPartial = 4,  // a share of K: fp32 sums [share][M, N]
};

struct Product {
  const uint8_t* a;
  const uint8_t* b;
  const float* a_scales;  // [stage][a_rows]
  const float* b_scales;  // block row n / 128 (square) or row n (rows), and stage, at these pitches
  int64_t lda, ldb;       // bytes from a row to the next
  int64_t M;
  int32_t N;
  int64_t K;
  int64_t a_rows, sb_row, sb_stage;
  void* out = nullptr;
  float* aux = nullptr;
  int64_t m_first = 0, m_end = 0;  // set by a launch: the rows it computes
  // experts: the buckets (see moe_w4a16_align) of blocks as high as the tile, and the pairs;
  // B and its scales are each expert's after the other
  const int32_t* sorted = nullptr;
  const int32_t* block_expert = nullptr;
  const int32_t* n_padded = nullptr;
  int64_t pairs = 0;
  int32_t top_k = 1;
};
// How a product is cut (fp8_plan.cpp): the tile (0: 128 x 128, 1: 128 x 256, 2: 256 x 256, 3: 64
// x 64), its work-groups, and for tiles 0 and 3 the shares of K, `share` stages each. wide: fp32
// results, which tile 2 has no registers for; rows: B in 1 x 128 blocks.
struct Cut {
  int tile = 0, shares = 1, share = 1;
  int64_t groups = 0;
  double time = 0;  // estimate, microseconds
};
Cut cut_of(bool wide, bool rows, int64_t M, int64_t N, int64_t K);
// A product is one launch (with its join, for shares) of all rows, or two: the first rows in whole
// rounds of the largest tile, and the rest.
struct Plan {
  int64_t first = 0;  // rows of the first of two launches, 0: there is one
  Cut whole, rest;    // of the first or all rows, without shares where there are two; of the rest
  double time = 0;
};
Plan plan_of(bool wide, bool rows, int64_t M, int64_t N, int64_t K);
double rows_time(int64_t M, int64_t N, int64_t K);  // of the few-row kernel on codes
// Bytes of the shares' sums (`split`, 16-byte aligned)
size_t product_workspace(bool wide, bool rows, int64_t M, int32_t N, int64_t K);
hipError_t launch_product(Mode mode, Epilogue epilogue, const Product& p, void* split,
                          hipStream_t stream);
// The same for a few rows of A (fp8_rows.hip): codes, or bf16 (experts' h: fp32) rows that are
// quantised on the way; B's scales square, all of B (an expert's) below 2 GiB. rows_fit: whether
// the kernel takes the sizes (experts: M = kFewRows, N of W13's 2 I rows or W2's).
enum Source { kCodes = 0, kBf16 = 1, kF32 = 2 };
constexpr int kMostRows = 16, kFewRows = 4;  // of codes; to quantise, and of an experts' bucket
bool rows_fit(Source source, int64_t M, int64_t N, int64_t K);
// A work-group of theirs: the waves, the bytes of a wave's stage (16 weight rows), the stages in
// flight, and the columns of a slice
constexpr int kRowsWaves = 8, kRowsSlot = 16 * kBlock, kRowsStages = 6, kExpertsStages = 3;
constexpr int rows_step(Epilogue epilogue) { return epilogue == kSwiglu ? 8 : 16; }
// Its LDS beside the ring: `rows` quantised rows (fresh; 16 of them at one offset lie in distinct
// bank groups), the scales of A and of B by stage, and (fresh) at rows_sums_at the waves' sums of
// each slice
__host__ __device__ inline int rows_code_stride(int64_t K) {
  return (int)((K + 255) / 256 * 256 + 16);
}
__host__ __device__ inline int64_t rows_sums_at(bool fresh, int64_t rows, int64_t K) {
  return (fresh ? rows * rows_code_stride(K) : 0) + (4 * (rows + 2) * blocks_of(K) + 15) / 16 * 16;
}
int64_t rows_extra(bool fresh, int64_t rows, int64_t K, int slices);
// Slices of an experts' work-group (N, K: of the product)
int experts_slices(Epilogue epilogue, int64_t N, int64_t K, int64_t buckets);
hipError_t launch_rows(Source source, Epilogue epilogue, const Product& p, hipStream_t stream);
// kSwiglu: from x bf16 [T, H], h fp32 [bucket rows, I]; kPairs: from that h
hipError_t launch_experts_rows(Epilogue epilogue, const Product& p, int64_t buckets,
                               hipStream_t stream);
// The experts' products (kSwiglu, kPairs) over buckets of kBigRows rows; M: the most bucket
// rows, a launch's of at most kMaxGroups tiles
constexpr int kBigRows = 256;
hipError_t launch_experts(Epilogue epilogue, const Product& p, hipStream_t stream);
// kPairs: column tiles that a work-group takes in turn, tm blocks by tn tiles (the device knows the
// blocks): as many as cost no round of work-groups on 256 CUs more than one does
__host__ __device__ inline int experts_span(int64_t tm, int64_t tn) {
  const int64_t rounds = (tm * tn + 255) / 256;
  int span = 1;
  for (int more = 2; more <= 4; more *= 2)
    if ((tm * ((tn + more - 1) / more) + 255) / 256 * more * 32 <= rounds * 33) span = more;
  return span;
}

}  // namespace fp8
