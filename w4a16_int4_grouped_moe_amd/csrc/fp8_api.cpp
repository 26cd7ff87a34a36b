// fp8_api.cpp -- host side of include/moe_fp8.h: argument checks, workspace
// layout and launch sequences. Every check runs before the first launch.
#include <algorithm>
#include <initializer_list>

#include "../../include/moe_fp8.h"
#include "fp8_internal.h"
#include "internal.h"

namespace {

using fp8::blocks_of;
using fp8::kBlock;
using fp8::Product;

constexpr int32_t kMaxWidth = 1 << 20;
constexpr int64_t kMaxRows = 0x7fffff00;  // whole 256-row tiles below 2^31

size_t region(int64_t bytes) { return ((size_t)bytes + 255) / 256 * 256; }
bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }
int done(hipError_t e) { return e == hipSuccess ? MOE_OK : moe::report_hip(e); }

int check_matrix(int64_t rows, int32_t width) {
  if (rows < 0 || rows > kMaxRows || width <= 0 || width > kMaxWidth || width % 16)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}
int check_product(int64_t rows, int32_t cols, int32_t width) {
  const int st = check_matrix(rows, width);
  if (st != MOE_OK) return st;
  return cols <= 0 || cols > kMaxRows || cols % 8 ? MOE_ERR_SHAPE : MOE_OK;
}
// The gradients also sum over rows and over cols
int check_gradients(int64_t rows, int32_t cols, int32_t width) {
  const int st = check_product(rows, cols, width);
  if (st != MOE_OK) return st;
  return rows > kMaxWidth || cols > kMaxWidth ? MOE_ERR_SHAPE : MOE_OK;
}
int check_type(int32_t type) {
  return type < MOE_TYPE_BF16 || type > MOE_TYPE_FP32 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
int check_block(int32_t block) {
  return block != MOE_FP8_ROW_BLOCKS && block != MOE_FP8_SQUARE_BLOCKS ? MOE_ERR_UNSUPPORTED
                                                                       : MOE_OK;
}

// every pointer given, then every one aligned (tensors 16 bytes, scales 4)
int check_pointers(std::initializer_list<const void*> tensors,
                   std::initializer_list<const void*> scales) {
  for (const void* p : tensors)
    if (!p) return MOE_ERR_NULL;
  for (const void* p : scales)
    if (!p) return MOE_ERR_NULL;
  for (const void* p : tensors)
    if (!aligned(p, 16)) return MOE_ERR_ALIGNMENT;
  for (const void* p : scales)
    if (!aligned(p, 4)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}
int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return MOE_OK;
  if (!ws) return MOE_ERR_NULL;
  if (!aligned(ws, 16)) return MOE_ERR_ALIGNMENT;
  return have < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

// A quantised matrix in a workspace, 1 x 128 blocks: codes, then scales
struct Quantized {
  int64_t pitch;  // bytes of a row
  size_t codes, scales;
  Quantized(int64_t rows, int64_t width, bool padded = false)
      : pitch(padded ? kBlock * blocks_of(width) : width),
        codes(region(rows * pitch)),
        scales(region(4 * blocks_of(width) * rows)) {}
  size_t bytes() const { return codes + scales; }
};

// Which kernel a product takes: few rows, quantised on the way where they are bf16 and four at
// most, or by a launch ahead; or tiles. Sizes alone choose between few rows and tiles, so that a
// bf16 operand and its codes give the same bits: up to four rows the few-row kernel may be
// kAhead microseconds longer by the estimates, the launch that tiles of a bf16 operand need. Codes
// alone, which do not need it, in few rows and in tiles, microseconds: 1 x 256 x 8192 6.9 and 13.1, 4 x
// 1024 x 8192 7.9 and 12.4, 1 x 7168 x 7168 15.3 and 17.7, 4 x 7168 x 2048 10.0 and 9.7, 4 x 7168 x 1024
// 8.8 and 6.8; bf16 at the last 9.4 and 8.9.
constexpr double kAhead = 3.0;
enum Path { kFew, kFewPrepared, kTiled };
Path path_of(int64_t rows, int32_t cols, int32_t width, bool quantize, bool square, bool wide) {
  if (!square || !fp8::rows_fit(fp8::kCodes, rows, cols, width)) return kTiled;
  const bool fresh = fp8::rows_fit(fp8::kBf16, rows, cols, width);
  const double tiled = fp8::plan_of(wide, false, rows, cols, width).time;
  if (fp8::rows_time(rows, cols, width) >= tiled + (fresh ? kAhead : 0)) return kTiled;
  return quantize && !fresh ? kFewPrepared : kFew;
}

// The shares' sums of a product, of either type of result and either kind of B
size_t split_of(int64_t rows, int32_t cols, int64_t width) {
  size_t most = 0;
  for (int kind = 0; kind < 4; ++kind)
    most = std::max(most, fp8::product_workspace(kind & 1, kind & 2, rows, cols, width));
  return region(most);
}

// ---- the gradients' workspace ----
struct Gradients {
  Quantized dout, dout_t, a_t;
  size_t weights;  // B transposed
  size_t split;    // of da's product, then of db's
  Gradients(int64_t rows, int32_t cols, int32_t width)
      : dout(rows, cols, true),
        dout_t(cols, rows, true),
        a_t(width, rows, true),
        weights(region((int64_t)width * kBlock * blocks_of(cols))),
        split(std::max(split_of(rows, width, dout.pitch), split_of(cols, width, dout_t.pitch))) {}
  size_t bytes() const { return dout.bytes() + weights + dout_t.bytes() + a_t.bytes() + split; }
};

// ---- the experts ----
constexpr int64_t kAlignMultiMin = 8192;  // pairs that many work-groups bucket

int check_experts(const moe_fp8_experts_problem* p) {
  if (!p) return MOE_ERR_NULL;
  if (p->num_tokens < 0 || p->hidden <= 0 || p->inter <= 0 || p->hidden % kBlock ||
      p->inter % kBlock || p->hidden > kMaxWidth || p->inter > kMaxWidth || p->num_experts <= 0 ||
      p->top_k <= 0 || p->top_k > MOE_MAX_TOP_K || p->expert_base < 0 ||
      (int64_t)p->expert_base + p->num_experts > 0x7fffffff ||
      p->num_tokens > 0x3fffffff / p->top_k)
    return MOE_ERR_SHAPE;
  if (p->num_experts > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Rows of a bucket's block: a few where an expert has two pairs at most on average, for the
// kernels that stream weights; else a tile's. Measured with all experts local, microseconds with
// a few and with tiles: 48 experts at 7168/2048, 8 tokens (1.3 pairs) 280 and 321, 16 (2.7) 413
// and 376; 256 experts at 2048/1024, 64 tokens (2.0) 250 and 319, 128 (4.0) 334 and 369. How many
// pairs are local only the device knows, so that the rule counts them all, and takes tiles too
// early where few are: 48 of 384 experts here, 16 tokens (19 local pairs) 150 with a few rows and
// 176 with tiles, 64 (75) 325 and 352, 96 (102) 369 and 364.
int32_t block_of(const moe_fp8_experts_problem* p) {
  const int64_t P = p->num_tokens * p->top_k;
  if (P <= 2 * (int64_t)p->num_experts &&
      fp8::rows_fit(fp8::kBf16, fp8::kFewRows, 2 * (int64_t)p->inter, p->hidden) &&
      fp8::rows_fit(fp8::kBf16, fp8::kFewRows, p->hidden, p->inter))
    return fp8::kFewRows;
  return fp8::kBigRows;
}

struct Experts {
  int32_t block;
  int64_t pairs, blocks, rows;  // the most blocks and bucket rows
  size_t x, sorted, block_expert, n_padded, scratch, h, y, bytes;
  Quantized qx, qh;
  static int64_t most_blocks(const moe_fp8_experts_problem* p, int32_t block) {
    const int64_t P = p->num_tokens * p->top_k;
    return (P + std::min<int64_t>(P, p->num_experts) * (block - 1)) / block;
  }
  explicit Experts(const moe_fp8_experts_problem* p)
      : block(block_of(p)),
        pairs(p->num_tokens * p->top_k),
        blocks(most_blocks(p, block)),
        rows(blocks * block),
        qx(p->num_tokens, p->hidden),
        qh(rows, p->inter) {
    const bool few = block == fp8::kFewRows;  // quantises x and h on the way
    size_t at = 0;
    const auto take = [&](size_t n) {
      const size_t here = at;
      at += n;
      return here;
    };
    x = take(few ? 0 : qx.bytes());
    // the bucketing writes a block's padding whole, and needs no more than pairs + E (block - 1)
    sorted = take(region(4 * (pairs + std::min<int64_t>(pairs, p->num_experts) * (block - 1))));
    block_expert = take(region(4 * blocks));
    n_padded = take(region(16));
    scratch = take(pairs >= kAlignMultiMin
                       ? region(4 * moe::align_scratch_ints(pairs, p->num_experts))
                       : 0);
    h = take(few ? region(4 * rows * p->inter) : qh.bytes());
    y = take(region(4 * pairs * p->hidden));
    bytes = p->num_tokens ? at : 0;
  }
};

}  // namespace

extern "C" {

int moe_fp8_quantize(const void* x, int32_t type, int64_t rows, int32_t width, int32_t block,
                     uint8_t* codes, float* scales, void* stream) {
  int st = check_matrix(rows, width);
  if (st != MOE_OK || (st = check_type(type)) != MOE_OK || (st = check_block(block)) != MOE_OK)
    return st;
  if (rows == 0) return MOE_OK;
  if ((st = check_pointers({x, codes}, {scales})) != MOE_OK) return st;
  return done(
      fp8::launch_quantize(x, type, rows, width, block, codes, scales, (hipStream_t)stream));
}

int moe_fp8_dequantize(const uint8_t* codes, const float* scales, int64_t rows, int32_t width,
                       int32_t block, int32_t type, void* out, void* stream) {
  int st = check_matrix(rows, width);
  if (st != MOE_OK || (st = check_type(type)) != MOE_OK || (st = check_block(block)) != MOE_OK)
    return st;
  if (rows == 0) return MOE_OK;
  if ((st = check_pointers({codes, out}, {scales})) != MOE_OK) return st;
  return done(
      fp8::launch_dequantize(codes, scales, rows, width, block, type, out, (hipStream_t)stream));
}

int moe_fp8_matmul_workspace_size(int64_t rows, int32_t cols, int32_t width, int quantize,
                                  size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const int st = check_product(rows, cols, width);
  if (st != MOE_OK) return st;
  *bytes = rows ? (quantize ? Quantized(rows, width).bytes() : 0) + split_of(rows, cols, width) : 0;
  return MOE_OK;
}

int moe_fp8_matmul(const void* a, const float* a_scales, const uint8_t* b, const float* b_scales,
                   int32_t b_block, int64_t rows, int32_t cols, int32_t width, int32_t out_type,
                   void* out, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int st = moe_fp8_matmul_workspace_size(rows, cols, width, !a_scales, &need);
  if (st != MOE_OK || (st = check_block(b_block)) != MOE_OK) return st;
  if (out_type != MOE_TYPE_BF16 && out_type != MOE_TYPE_FP32) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if ((st = check_pointers({a, b, out}, {b_scales})) != MOE_OK) return st;
  if (!aligned(a_scales, 4)) return MOE_ERR_ALIGNMENT;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MOE_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* split = (uint8_t*)workspace;
  const bool square = b_block == MOE_FP8_SQUARE_BLOCKS, quantize = !a_scales;
  const Path path = path_of(rows, cols, width, quantize, square, out_type != MOE_TYPE_BF16);
  if (quantize && path != kFew) {
    const Quantized q(rows, width);
    uint8_t* codes = split;
    float* scales = (float*)(codes + q.codes);
    split += q.bytes();
    const hipError_t e =
        fp8::launch_quantize(a, MOE_TYPE_BF16, rows, width, MOE_FP8_ROW_BLOCKS, codes, scales, s);
    if (e != hipSuccess) return done(e);
    a = codes;
    a_scales = scales;
  }
  Product d{(const uint8_t*)a, b, a_scales, b_scales, width, width, rows, cols, width};
  d.a_rows = rows;
  d.sb_row = square ? blocks_of(width) : 1;
  d.sb_stage = square ? 1 : cols;
  d.out = out;
  if (path != kTiled)
    return done(fp8::launch_rows(quantize && path == kFew ? fp8::kBf16 : fp8::kCodes,
                                 out_type == MOE_TYPE_BF16 ? fp8::kStoreBf16 : fp8::kStoreF32, d,
                                 s));
  return done(fp8::launch_product(square ? fp8::kSquare : fp8::kRowScales,
                                  out_type == MOE_TYPE_BF16 ? fp8::kStoreBf16 : fp8::kStoreF32, d,
                                  split, s));
}

int moe_fp8_matmul_backward_workspace_size(int64_t rows, int32_t cols, int32_t width,
                                           size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const int st = check_gradients(rows, cols, width);
  if (st != MOE_OK) return st;
  const Gradients g(rows, cols, width);
  *bytes = rows ? g.bytes() : 0;
  return MOE_OK;
}

int moe_fp8_matmul_backward(const void* dout, const void* a, const uint8_t* b,
                            const float* b_scales, int64_t rows, int32_t cols, int32_t width,
                            int32_t out_type, void* da, void* db, void* workspace,
                            size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int st = moe_fp8_matmul_backward_workspace_size(rows, cols, width, &need);
  if (st != MOE_OK) return st;
  if (out_type != MOE_TYPE_BF16 && out_type != MOE_TYPE_FP32) return MOE_ERR_UNSUPPORTED;
  if (!da && !db) return MOE_ERR_NULL;
  if (!aligned(da, 16) || !aligned(db, 16)) return MOE_ERR_ALIGNMENT;
  hipStream_t s = (hipStream_t)stream;
  const fp8::Epilogue store = out_type == MOE_TYPE_BF16 ? fp8::kStoreBf16 : fp8::kStoreF32;
  hipError_t e = hipSuccess;
  if (rows > 0) {
    if ((st = check_pointers({dout}, {})) != MOE_OK) return st;
    if (da && (st = check_pointers({b}, {b_scales})) != MOE_OK) return st;
    if (db && (st = check_pointers({a}, {})) != MOE_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, need)) != MOE_OK) return st;
  }
  if (rows == 0) {
    if (db) e = fp8::launch_clear(db, (int64_t)cols * width * (out_type == MOE_TYPE_BF16 ? 2 : 4), s);
    return done(e);
  }
  const Gradients g(rows, cols, width);
  uint8_t* const dout_codes = (uint8_t*)workspace;
  uint8_t* const b_t = dout_codes + g.dout.bytes();
  uint8_t* const dout_t = b_t + g.weights;
  uint8_t* const a_t = dout_t + g.dout_t.bytes();
  uint8_t* const split = a_t + g.a_t.bytes();
  fp8::Prepare q{dout, a, b, rows, cols, width};
  float* const dout_scales = (float*)(dout_codes + g.dout.codes);
  float* const dout_t_scales = (float*)(dout_t + g.dout_t.codes);
  float* const a_t_scales = (float*)(a_t + g.a_t.codes);
  if (da) q.b_t = b_t, q.dout_codes = dout_codes, q.dout_scales = dout_scales;
  if (db)
    q.dout_t = dout_t, q.dout_t_scales = dout_t_scales, q.a_t = a_t, q.a_t_scales = a_t_scales;
  e = fp8::launch_prepare(q, s);
  if (da && e == hipSuccess) {
    Product d{dout_codes, b_t, dout_scales, b_scales, g.dout.pitch, kBlock * blocks_of(cols),
              rows, width, g.dout.pitch};
    d.a_rows = rows;
    d.sb_row = 1;
    d.sb_stage = blocks_of(width);
    d.out = da;
    e = fp8::launch_product(fp8::kSquare, store, d, split, s);
  }
  if (db && e == hipSuccess) {
    Product d{dout_t, a_t, dout_t_scales, a_t_scales, g.dout_t.pitch, g.a_t.pitch,
              cols, width, g.dout_t.pitch};
    d.a_rows = cols;
    d.sb_row = 1;
    d.sb_stage = width;
    d.out = db;
    e = fp8::launch_product(fp8::kRowScales, store, d, split, s);
  }
  return done(e);
}

int moe_fp8_experts_workspace_size(const moe_fp8_experts_problem* p, size_t* bytes) {
  if (!p || !bytes) return MOE_ERR_NULL;
  const int st = check_experts(p);
  if (st != MOE_OK) return st;
  const Experts w(p);
  // what the kernels address by 32-bit offsets: x's codes, and tiles in one launch
  const int64_t across = std::max<int64_t>(p->inter / kBlock, (p->hidden + 255) / 256);
  if (p->num_tokens * p->hidden > 0x7fffffff || w.rows > kMaxRows ||
      w.blocks > fp8::kMaxGroups / across)
    return MOE_ERR_UNSUPPORTED;
  *bytes = w.bytes;
  return MOE_OK;
}

int moe_fp8_experts_forward(const void* x, const int32_t* topk_ids, const float* topk_weights,
                            const uint8_t* w13, const float* w13_scales, const uint8_t* w2,
                            const float* w2_scales, void* out, const moe_fp8_experts_problem* p,
                            void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int st = moe_fp8_experts_workspace_size(p, &need);
  if (st != MOE_OK || p->num_tokens == 0) return st;
  st = check_pointers({x, w13, w2, out}, {topk_ids, topk_weights, w13_scales, w2_scales});
  if (st != MOE_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MOE_OK) return st;
  const Experts w(p);
  const int64_t T = p->num_tokens;
  const int32_t H = p->hidden, I = p->inter, E = p->num_experts;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* ws = (uint8_t*)workspace;
  uint8_t *xc = ws + w.x, *hc = ws + w.h;
  float *xs = (float*)(xc + w.qx.codes), *hs = (float*)(hc + w.qh.codes);
  int32_t *sorted = (int32_t*)(ws + w.sorted), *blocks = (int32_t*)(ws + w.block_expert);
  int32_t* n_padded = (int32_t*)(ws + w.n_padded);
  const bool few = w.block == fp8::kFewRows;
  hipError_t e = hipSuccess;
  if (!few) e = fp8::launch_quantize(x, MOE_TYPE_BF16, T, H, MOE_FP8_ROW_BLOCKS, xc, xs, s);
  if (e != hipSuccess) return done(e);
  if (w.pairs >= kAlignMultiMin)
    e = moe::launch_align_multi(topk_ids, w.pairs, E, p->expert_base, w.block, sorted, blocks,
                                n_padded, (int32_t*)(ws + w.scratch), s);
  else
    e = moe::launch_align(topk_ids, w.pairs, E, p->expert_base, w.block, sorted, blocks, n_padded,
                          s);
  if (e != hipSuccess) return done(e);
  Product up{xc, w13, xs, w13_scales, H, H, w.rows, I, H};
  up.a_rows = T;
  up.sb_row = H / kBlock;
  up.sb_stage = 1;
  up.out = hc;
  up.aux = hs;
  up.sorted = sorted;
  up.block_expert = blocks;
  up.n_padded = n_padded;
  up.pairs = w.pairs;
  up.top_k = p->top_k;
  if (few) up.a = (const uint8_t*)x;
  e = few ? fp8::launch_experts_rows(fp8::kSwiglu, up, w.blocks, s)
          : fp8::launch_experts(fp8::kSwiglu, up, s);
  if (e != hipSuccess) return done(e);
  Product down = up;
  down.a = hc;
  down.b = w2;
  down.a_scales = hs;
  down.b_scales = w2_scales;
  down.lda = down.ldb = down.K = I;
  down.N = H;
  down.a_rows = w.rows;
  down.sb_row = I / kBlock;
  down.out = ws + w.y;
  down.aux = nullptr;
  e = few ? fp8::launch_experts_rows(fp8::kPairs, down, w.blocks, s)
          : fp8::launch_experts(fp8::kPairs, down, s);
  if (e != hipSuccess) return done(e);
  return done(moe::launch_combine((const float*)(ws + w.y), nullptr, topk_ids, topk_weights,
                                  (uint16_t*)out, T, H, p->top_k, E, p->expert_base, s));
}

}  // extern "C"
