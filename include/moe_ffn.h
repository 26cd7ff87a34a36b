/*
 * moe_ffn.h -- C ABI of the gated feed-forward block (forward and backward)
 * and of the MXFP4 operators beside the W4A16 MoE layer (MI355X, gfx950).
 *
 * The block is the layer's shared expert on its own, bf16:
 *
 *   g = x W1^T,  u = x W3^T,  W1 = w13[0:I], W3 = w13[I:2I]
 *   h = silu(g) * u           rounded once to bf16
 *   out = h W2^T              rounded once to bf16; sums in fp32
 *
 * MXFP4: along a row, each block of 32 values v is one power-of-two scale and
 * 32 e2m1 codes (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3,
 * 4, 6):
 *
 *   e = floor(log2(max |v|)) - 2, stored as the byte e + 127, at least 0
 *       (a block of zeros: 0)
 *   code = nearest e2m1 of v * 2^-e, ties to the even code, above 6 to 6
 *   a block that holds an infinity or a NaN: byte 255, codes 0; its values
 *   read back as NaN
 *
 * Codes are packed two a byte along the row, the even input in the low four
 * bits: codes uint8 [rows, width/2], scales uint8 [rows, width/32].
 *
 * Conventions are moe_w4a16.h's: dense row-major device tensors, 16-byte
 * aligned (scales need no alignment); the caller owns every buffer and the
 * workspace; nothing is allocated or kept, the host never waits, launches go
 * to `stream` on the current device and may be captured into a HIP graph;
 * calls that share a workspace (two captured graphs, too) must not overlap;
 * every argument error is found on the host before any launch and returned
 * as one of moe_w4a16.h's status codes. Outputs must not overlap inputs.
 * Results do not depend on anything but the inputs: no atomics, and the same
 * call gives the same bits.
 *
 * Limits: hidden, inter and width at most 2^20; hidden and inter multiples of
 * 8 (bf16) or 32 (MXFP4), cols a multiple of 8, width a multiple of 32;
 * num_tokens, rows and cols at most 2^31 - 256.
 */
#ifndef MOE_FFN_H
#define MOE_FFN_H

#include "moe_w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types of a tensor argument */
#define MOE_TYPE_BF16 0
#define MOE_TYPE_FP16 1
#define MOE_TYPE_FP32 2

/* what a workspace is for */
#define MOE_FFN_FORWARD 0
#define MOE_FFN_BACKWARD 1
#define MOE_FFN_FORWARD_MXFP4 2

/* Sizes of a feed-forward block (host struct, read during the call only). */
typedef struct {
  int64_t num_tokens; /* T >= 0 */
  int32_t hidden;     /* H */
  int32_t inter;      /* I */
} moe_ffn_problem;

/* Bytes of workspace of one call (host only). `pass`: MOE_FFN_*. */
int moe_ffn_workspace_size(const moe_ffn_problem *p, int pass, size_t *bytes);

/*
 * out bf16 [T, H] from x bf16 [T, H], w13 bf16 [2I, H], w2 bf16 [H, I].
 * gate_up: NULL, or fp32 [T, 2I] that receives [g, u] for the backward pass.
 * T == 0 is a successful no-op.
 */
int moe_ffn_forward(const void *x, const void *w13, const void *w2, void *out, float *gate_up,
                    const moe_ffn_problem *p, void *workspace, size_t workspace_bytes,
                    void *stream);

/*
 * Gradients of sum(out * dout) with respect to x, w13 and w2, all bf16: dx
 * [T, H], dw13 [2I, H], dw2 [H, I], written (not added to). gate_up: what
 * moe_ffn_forward wrote for the same x and w13. The gradients of g and u and
 * the recomputed h are each rounded once to bf16 before the last products.
 * dx, or both of dw13 and dw2, may be NULL: that part is then not computed (and
 * the sums of the other may be added in another order).
 * T == 0 clears dw13 and dw2.
 */
int moe_ffn_backward(const void *dout, const void *x, const float *gate_up, const void *w13,
                     const void *w2, void *dx, void *dw13, void *dw2, const moe_ffn_problem *p,
                     void *workspace, size_t workspace_bytes, void *stream);

/* x [rows, width] of `type` -> codes, scales. rows == 0 is a no-op. */
int moe_mxfp4_quantize(const void *x, int32_t type, int64_t rows, int32_t width, uint8_t *codes,
                       uint8_t *scales, void *stream);

/* The values of codes and scales, rounded once to `type`: out [rows, width]. */
int moe_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int32_t width,
                         int32_t type, void *out, void *stream);

/* Bytes of workspace of moe_mxfp4_matmul; quantize: whether a is bf16. */
int moe_mxfp4_matmul_workspace_size(int64_t rows, int32_t cols, int32_t width, int quantize,
                                    size_t *bytes);

/*
 * out [rows, cols] = A B^T, fp32 sums, rounded once to out_type (MOE_TYPE_BF16
 * or MOE_TYPE_FP32). B: codes and scales of [cols, width]. A [rows, width]:
 * codes and scales, or bf16 with a_scales NULL, which is quantised as by
 * moe_mxfp4_quantize. rows == 0 is a no-op.
 */
int moe_mxfp4_matmul(const void *a, const uint8_t *a_scales, const uint8_t *b,
                     const uint8_t *b_scales, int64_t rows, int32_t cols, int32_t width,
                     int32_t out_type, void *out, void *workspace, size_t workspace_bytes,
                     void *stream);

/*
 * The block on MXFP4 weights: w13 codes/scales of [2I, H], w2 of [H, I]. x
 * (bf16) and h (from its fp32 value) are quantised to MXFP4 on the way.
 * T == 0 is a no-op.
 */
int moe_mxfp4_ffn_forward(const void *x, const uint8_t *w13, const uint8_t *w13_scales,
                          const uint8_t *w2, const uint8_t *w2_scales, void *out,
                          const moe_ffn_problem *p, void *workspace, size_t workspace_bytes,
                          void *stream);

#ifdef __cplusplus
}
#endif
#endif
