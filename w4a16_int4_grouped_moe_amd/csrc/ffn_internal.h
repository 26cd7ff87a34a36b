// ffn_internal.h -- what the feed-forward and MXFP4 entry points share.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ffn {

// What a product's epilogue does with its tile. "N" below is the product's
// column count (gate_up: the intermediate width, each column being a gate and
// an up column of the weight matrix).
enum Epilogue {
  kStoreBf16 = 0,   // out bf16 [M, N]
  kStoreF32 = 1,    // out fp32 [M, N]
  kSwiglu = 2,      // out bf16 h [M, N]; aux fp32 [M, 2N] pre-activations or NULL
  kSwigluMx = 3,    // out e2m1 codes of h [M, N/2], aux its scale bytes (scale_stride(N) a row)
  kSwigluGrad = 4,  // the product is dh: aux fp32 [M, 2N] pre-activations (read),
                    // out bf16 [M, 2N] their gradients, out2 bf16 h [M, N]
  kSwigluF32 = 5,   // out fp32 h [M, N]
};

// D[m, n] = sum_k A(m, k) B(n, k). An operand is "K contiguous" (element
// (r, k) at r * ld + k) or "row contiguous" (at k * ld + r); which one is a
// template parameter of the kernel (see Layout).
enum Layout { kNT = 0, kNN = 1, kTN = 2 };  // A/B: KC/KC, KC/RC, RC/RC

// The products read scale bytes eight at a time (one stage of K): each row's
// scales are padded to whole stages, and rows start at multiples of 8 bytes.
// The padding holds 127 (the scale 1; the codes there are 0).
__host__ __device__ inline int64_t scale_stride(int64_t K) { return (K / 32 + 7) / 8 * 8; }

struct Product {
  const void* a;
  const void* b;
  const uint8_t* a_scales = nullptr;  // MXFP4: e8m0 bytes, rows of scale_stride(K)
  const uint8_t* b_scales = nullptr;
  int64_t lda, ldb;  // bytes from one row (KC) or one k (RC) to the next
  int64_t M;
  int32_t N;
  int64_t K;
  void* out = nullptr;
  void* out2 = nullptr;
  void* aux = nullptr;
};

// bf16 operands
hipError_t launch_product(Layout layout, Epilogue epilogue, const Product& p, hipStream_t stream);
// MXFP4 operands, both K contiguous; K a multiple of 32
hipError_t launch_product_mx(Epilogue epilogue, const Product& p, hipStream_t stream);

// The same products for a few rows (ffn_small.hip), both operands K contiguous
// and dense. A: as the product takes it, or rows to be quantised to MXFP4.
// Here a row's scales are K/32 bytes, at any address. rows_fit: whether the
// kernel takes the problem (at most 16 rows, B below 2 GiB, a quantised A that
// fits LDS).
enum AType { kAAsIs = 0, kABf16 = 1, kAF32 = 2 };
bool rows_fit(const Product& p, bool mx, AType a, bool paired);
hipError_t launch_rows(Epilogue epilogue, const Product& p, hipStream_t stream);
hipError_t launch_rows_mx(Epilogue epilogue, AType a, const Product& p, hipStream_t stream);

// x [rows, width] (type: MOE_TYPE_*) -> e2m1 codes [rows, width/2], scales
// [rows, width/32], or padded: rows of scale_stride(width)
hipError_t launch_mx_quantize(const void* x, int32_t type, int64_t rows, int32_t width,
                              uint8_t* codes, uint8_t* scales, bool padded, hipStream_t stream);
// Two matrices' scales [rows, width/32] copied into padded rows (either may be
// NULL with 0 rows)
hipError_t launch_mx_pad_scales(const uint8_t* s0, int64_t rows0, uint8_t* out0,
                                const uint8_t* s1, int64_t rows1, uint8_t* out1, int32_t width,
                                hipStream_t stream);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                int32_t width, int32_t type, void* out, hipStream_t stream);

}  // namespace ffn
