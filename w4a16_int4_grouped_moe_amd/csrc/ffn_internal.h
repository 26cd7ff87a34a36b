// ffn_internal.h -- what the feed-forward and MXFP4 entry points share.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace ffn {

// What a product's epilogue does with its tile. "N" below is the product's
// column count (gate_up: the intermediate width, each column being a gate and
// an up column of the weight matrix).
enum Epilogue {
  kStoreBf16 = 0,   // out bf16 [M, N]
  kStoreF32 = 1,    // out fp32 [M, N]
  kSwiglu = 2,      // out bf16 h [M, N]; aux fp32 [M, 2N] pre-activations or NULL
  kSwigluMx = 3,    // out e2m1 codes of h [M, N/2], aux its scale bytes by stage
  kSwigluGrad = 4,  // the product is dh: aux fp32 [M, 2N] pre-activations (read),
                    // out bf16 [M, 2N] their gradients, out2 bf16 h [M, N]
  kSwigluF32 = 5,   // out fp32 h [M, N]
  kPartial = 6,     // a share of K: fp32 sums [share][M, N] in out
  kPartialPaired = 7,  // fp32 gate and up sums [share][M, 2N]
  kStoreOrSums = 8,    // as kStoreBf16, or where aux is given fp32 sums [share][M, N] there
};

// D[m, n] = sum_k A(m, k) B(n, k). An operand is "K contiguous" (element
// (r, k) at r * ld + k) or "row contiguous" (at k * ld + r); which one is a
// template parameter of the kernel (see Layout).
enum Layout { kNT = 0, kNN = 1, kTN = 2 };  // A/B: KC/KC, KC/RC, RC/RC

// The tiled products read scales a stage of K (8 blocks) at a time, all rows of
// a tile together: [stage][row][8 bytes], rows padded to an even number, the
// last stage's missing blocks with any finite scale (their codes are 0).
__host__ __device__ inline int64_t scale_stages(int64_t K) { return (K + 255) / 256; }
__host__ __device__ inline int64_t scale_rows(int64_t rows) { return (rows + 1) / 2 * 2; }
__host__ __device__ inline int64_t scale_bytes(int64_t rows, int64_t K) {
  return 8 * scale_rows(rows) * scale_stages(K);
}

struct Product {
  const void* a;
  const void* b;
  const uint8_t* a_scales = nullptr;  // MXFP4: e8m0 bytes by stage, scale_rows(M) and
                                      // scale_rows(rows of b) a stage
  const uint8_t* b_scales = nullptr;
  int64_t lda, ldb;  // bytes from one row (KC) or one k (RC) to the next
  int64_t M;
  int32_t N;
  int64_t K;
  void* out = nullptr;
  void* out2 = nullptr;
  void* aux = nullptr;
  int64_t m_first = 0, m_end = 0;  // set by a launch: the rows it computes
};

// bf16 operands. split: workspace of product_workspace bytes (16-byte aligned).
hipError_t launch_product(Layout layout, Epilogue epilogue, const Product& p, void* split,
                          hipStream_t stream);
// MXFP4 operands, both K contiguous; K a multiple of 32
hipError_t launch_product_mx(Epilogue epilogue, const Product& p, void* split,
                             hipStream_t stream);

// How a tiled product is cut (ffn_plan.cpp): the tile (0: 128 x 128, 1: 128 x
// 256, 2: 256 x 256, 3: 64 x 64; half the columns where gate and up pair), its
// work-groups, and for tiles 0 and 3 the shares of K, `share` stages each.
struct Cut {
  int tile = 0, shares = 1, share = 1;
  int64_t groups = 0;
  double time = 0;  // estimate, microseconds
};
struct Plan {
  int64_t first = 0;  // rows of a first launch where there are two, or 0
  Cut whole, rest;    // whole: of the first rows, where there are two
  double time = 0;
};
Plan plan_of(Epilogue epilogue, int64_t M, int64_t N, int64_t K, Layout layout, bool mx);
// f(first row, end of the rows, cut) for each launch of a plan's tiles. One holds
// fewer than 2^32 lanes, 2^23 - 1 work-groups of 512: more tiles go row range by
// row range. (A row of tiles fits: N is at most 2^31 - 256, and 2^20 where gate
// and up pair. Cuts with shares of K have 1024 work-groups at most.)
constexpr int64_t kMaxGroups = 0x7fffff;
template <typename F>
hipError_t each_launch(const Plan& plan, int64_t M, F&& f) {
  constexpr int64_t tile_rows[] = {128, 128, 256, 64};
  const int64_t split = plan.first ? plan.first : M;
  for (int part = 0; part < (plan.first ? 2 : 1); ++part) {
    Cut c = part ? plan.rest : plan.whole;
    const int64_t end = part ? M : split, size = tile_rows[c.tile];
    const int64_t across = c.groups / ((end - (part ? split : 0) + size - 1) / size);
    const int64_t most = kMaxGroups / across * size;
    for (int64_t m = part ? split : 0; m < end; m += most) {
      const int64_t m_end = std::min(m + most, end);
      c.groups = (m_end - m + size - 1) / size * across;
      const hipError_t e = f(m, m_end, c);
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}
// Bytes of the shares' sums (`split`), and the plan's time
size_t product_workspace(Layout layout, Epilogue epilogue, int64_t M, int32_t N, int64_t K,
                         bool mx);
double product_time(Layout layout, Epilogue epilogue, int64_t M, int32_t N, int64_t K, bool mx);

// The backward pass's last three products (dx: NN; dw13, dw2: TN; bf16 results)
// in one launch of 128 x 128 or 64 x 64 tiles, each with its own shares of K, and
// one that adds the sums: `together` where that is the faster way. sums: where in
// `split` (`bytes` in all) the sums of a product with shares lie.
struct GradientsPlan {
  bool together = false;
  Cut cut[3];
  size_t sums[3] = {}, bytes = 0;
};
GradientsPlan gradients_plan(int64_t tokens, int64_t hidden, int64_t inter);
hipError_t launch_gradients(const GradientsPlan& plan, const Product (&products)[3], void* split,
                            hipStream_t stream);

// The same products for a few rows (ffn_small.hip), both operands K contiguous
// and dense. A: as the product takes it, or rows to be quantised to MXFP4.
// Here a row's scales are K/32 bytes, at any address. rows_fit: whether the
// kernel takes the problem (at most 64 rows, 16 of bf16 to quantise; B below
// 2 GiB; a quantised A that fits LDS). The times are estimates in microseconds
// by which a call chooses.
enum AType { kAAsIs = 0, kABf16 = 1, kAF32 = 2 };
bool rows_fit(const Product& p, bool mx, AType a, bool paired);
double rows_time(const Product& p, bool mx, AType a, bool paired);
constexpr int kRowsThreads = 512;  // of a work-group
// LDS rows of an A quantised there: 16 rows at one offset lie in distinct banks
__host__ __device__ inline int rows_code_stride(int64_t K) {
  return (int)((K / 2 + 255) / 256 * 256 + 16);
}
__host__ __device__ inline int rows_byte_stride(int64_t K) {
  return (int)((K / 32 + 7) / 8 * 8 + 4);
}
hipError_t launch_rows(Epilogue epilogue, const Product& p, hipStream_t stream);
hipError_t launch_rows_mx(Epilogue epilogue, AType a, const Product& p, hipStream_t stream);

// x [rows, width] (type: MOE_TYPE_*) -> e2m1 codes [rows, width/2], scales [rows, width/32]
hipError_t launch_mx_quantize(const void* x, int32_t type, int64_t rows, int32_t width,
                              uint8_t* codes, uint8_t* scales, hipStream_t stream);
// What the tiled products need beforehand, in one launch: x bf16 (or NULL)
// quantised with its scales by stage, and up to two matrices' scales
// [rows, width/32] copied into that order (src NULL: none).
struct ScaleCopy {
  const uint8_t* src = nullptr;
  uint8_t* dst = nullptr;
  int64_t rows = 0;
  int32_t width = 0;
};
hipError_t launch_mx_prepare(const void* x, int64_t rows, int32_t width, uint8_t* codes,
                             uint8_t* scales, const ScaleCopy& s0, const ScaleCopy& s1,
                             hipStream_t stream);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                int32_t width, int32_t type, void* out, hipStream_t stream);

}  // namespace ffn
