// The host code of include/moe_fp8.h and include/moe_balance.h (csrc/fp8_api.cpp,
// csrc/fp8_plan.cpp, csrc/balance_api.cpp) over many sizes, with the launches
// replaced by checks: every array a launch is handed lies, with the size the
// kernel addresses, in a buffer of the caller or in the workspace of exactly the
// size the library asked for; cuts cover their product. No GPU.
#include <cstdio>
#include <vector>

#include "balance_internal.h"
#include "fp8_internal.h"
#include "internal.h"
#include "moe_balance.h"
#include "moe_fp8.h"

namespace {
struct Buffer {
  const char* at;
  size_t bytes;
};
std::vector<Buffer> buffers;
int failed = 0, launches = 0, cases = 0;
char* next_address = (char*)0x100000000000;

// an address range of its own; nothing of it is touched
void* buffer(size_t bytes) {
  char* at = next_address;
  next_address += (bytes + 4096) / 4096 * 4096 + 4096;
  buffers.push_back({at, bytes});
  return at;
}
void need(const void* p, int64_t bytes, const char* what) {
  if (bytes == 0) return;
  const char* c = static_cast<const char*>(p);
  for (const Buffer& b : buffers)
    if (bytes > 0 && c >= b.at && c + bytes <= b.at + b.bytes) return;
  std::fprintf(stderr, "%s: %lld bytes at %p outside every buffer\n", what, (long long)bytes, p);
  ++failed;
}
void expect(bool ok, const char* what) {
  if (!ok) std::fprintf(stderr, "failed: %s\n", what), ++failed;
}
int64_t row_scales(int64_t rows, int64_t width) { return 4 * rows * fp8::blocks_of(width); }
int64_t span(int64_t rows, int64_t ld, int64_t K) { return rows ? (rows - 1) * ld + K : 0; }

void operands(const fp8::Product& p, bool rows_mode, int64_t b_rows) {
  need(p.a, span(p.M, p.lda, p.K), "a");
  need(p.b, span(b_rows, p.ldb, p.K), "b");
  const int64_t stages = fp8::blocks_of(p.K);
  need(p.a_scales, 4 * ((stages - 1) * p.a_rows + p.M), "a's scales");
  const int64_t last = rows_mode ? b_rows - 1 : (b_rows - 1) / 128;
  need(p.b_scales, 4 * (last * p.sb_row + (stages - 1) * p.sb_stage + 1), "b's scales");
}
}  // namespace

namespace fp8 {
hipError_t launch_quantize(const void* x, int32_t type, int64_t rows, int32_t width, int32_t block,
                           uint8_t* codes, float* scales, hipStream_t) {
  ++launches;
  need(x, rows * width * (type == MOE_TYPE_FP32 ? 4 : 2), "x");
  need(codes, rows * width, "codes");
  need(scales, block == 1 ? row_scales(rows, width) : 4 * blocks_of(rows) * blocks_of(width), "scales");
  return hipSuccess;
}
hipError_t launch_dequantize(const uint8_t* codes, const float* scales, int64_t rows, int32_t width,
                             int32_t block, int32_t type, void* out, hipStream_t) {
  ++launches;
  need(out, rows * width * (type == MOE_TYPE_FP32 ? 4 : 2), "out");
  need(codes, rows * width, "codes");
  need(scales, block == 1 ? row_scales(rows, width) : 4 * blocks_of(rows) * blocks_of(width), "scales");
  return hipSuccess;
}
hipError_t launch_prepare(const Prepare& p, hipStream_t) {
  ++launches;
  expect(p.dout_codes || p.dout_t, "something of dout");
  need(p.dout, 2 * p.rows * p.cols, "dout");
  const int64_t high = 128 * blocks_of(p.rows);
  if (p.b_t) {
    need(p.b, (int64_t)p.cols * p.width, "b");
    need(p.b_t, p.width * 128 * blocks_of(p.cols), "b transposed");
  }
  if (p.dout_codes) {
    need(p.dout_codes, p.rows * 128 * blocks_of(p.cols), "dout's codes");
    need(p.dout_scales, row_scales(p.rows, p.cols), "dout's scales");
  }
  if (p.dout_t) {
    need(p.dout_t, p.cols * high, "dout transposed");
    need(p.dout_t_scales, row_scales(p.cols, p.rows), "its scales");
  }
  if (p.a_t) {
    need(p.a, 2 * p.rows * p.width, "a");
    need(p.a_t, p.width * high, "a transposed");
    need(p.a_t_scales, row_scales(p.width, p.rows), "its scales");
  }
  return hipSuccess;
}
hipError_t launch_clear(void* out, int64_t bytes, hipStream_t) {
  ++launches;
  expect(bytes % 16 == 0, "whole 16 bytes to clear");
  need(out, bytes, "cleared");
  return hipSuccess;
}
hipError_t launch_product(Mode mode, Epilogue e, const Product& p, void* split, hipStream_t) {
  ++launches;
  expect(mode == kSquare || mode == kRowScales, "mode");
  expect(e == kStoreBf16 || e == kStoreF32, "epilogue");
  operands(p, mode == kRowScales, p.N);
  need(p.out, p.M * p.N * (e == kStoreBf16 ? 2 : 4), "out");
  // tiles address their rows by 32-bit offsets
  expect(255 * p.lda + p.K <= 0x7fffffff && 255 * p.ldb + p.K <= 0x7fffffff, "a tile's offsets");
  const Plan plan = plan_of(e == kStoreF32, mode == kRowScales, p.M, p.N, p.K);
  expect(plan.first >= 0 && plan.first < p.M, "first rows");
  const int64_t high[] = {128, 128, 256, 64}, wide[] = {128, 256, 256, 64};
  const int64_t stages = blocks_of(p.K);
  for (int part = 0; part < (plan.first ? 2 : 1); ++part) {
    const Cut& c = part ? plan.rest : plan.whole;
    const int64_t rows = part ? p.M - plan.first : plan.first ? plan.first : p.M;
    expect(c.tile >= 0 && c.tile <= 3 && !(c.tile == 2 && e == kStoreF32), "tile");
    expect(c.groups == (rows + high[c.tile] - 1) / high[c.tile] * ((p.N + wide[c.tile] - 1) / wide[c.tile]), "groups");
    expect(c.shares == 1 ? c.share >= stages : (c.tile == 0 || c.tile == 3), "shares");
    expect((int64_t)c.shares * c.share >= stages && (int64_t)(c.shares - 1) * c.share < stages, "shares cover K");
    if (c.tile == 0 || c.tile == 3) expect(c.groups * c.shares <= 1024, "a launch");
    if (c.shares > 1) need(split, 4 * rows * p.N * c.shares, "sums");
    expect(part || !plan.first || c.shares == 1, "first rows without shares");
  }
  return hipSuccess;
}
bool rows_fit(Source source, int64_t M, int64_t N, int64_t K) {
  return M >= 1 && M <= (source == kCodes ? kMostRows : kFewRows) && N < (1 << 26) &&
         N * K <= 0x7fffffff && K <= 14000;
}
hipError_t launch_rows(Source source, Epilogue e, const Product& p, hipStream_t) {
  ++launches;
  expect(rows_fit(source, p.M, p.N, p.K), "few rows");
  need(p.out, p.M * p.N * (e == kStoreBf16 ? 2 : 4), "out");
  if (source == kCodes) return operands(p, false, p.N), hipSuccess;
  need(p.a, 2 * p.M * p.K, "a");
  need(p.b, p.N * p.K, "b");
  need(p.b_scales, 4 * blocks_of(p.N) * blocks_of(p.K), "b's scales");
  return hipSuccess;
}

int64_t experts_of = 0, tokens_of = 0;
void experts(Epilogue e, const Product& p, int64_t block, int64_t blocks, bool few) {
  const int64_t b_rows = e == kSwiglu ? 2 * (int64_t)p.N : p.N;
  need(p.sorted, 4 * blocks * block, "bucketed pairs");
  need(p.block_expert, 4 * blocks, "blocks");
  need(p.n_padded, 4, "count");
  need(p.b, experts_of * b_rows * p.ldb, "weights");
  need(p.b_scales, 4 * experts_of * (b_rows / 128) * p.sb_row, "weights' scales");
  const int64_t a_rows = e == kSwiglu ? tokens_of : blocks * block;
  need(p.a, a_rows * p.K * (few ? e == kSwiglu ? 2 : 4 : 1), "a");
  if (!few) {
    expect(p.a_rows == a_rows, "a's rows");
    need(p.a_scales, row_scales(a_rows, p.K), "a's scales");
  }
  if (e == kSwiglu) {
    need(p.out, blocks * block * p.N * (few ? 4 : 1), "h");
    if (!few) need(p.aux, row_scales(blocks * block, p.N), "h's scales");
  } else {
    need(p.out, 4 * p.pairs * p.N, "y");
  }
}
hipError_t launch_experts_rows(Epilogue e, const Product& p, int64_t buckets, hipStream_t) {
  ++launches;
  expect(buckets <= 65535, "buckets of a launch");
  experts(e, p, kFewRows, buckets, true);
  return hipSuccess;
}
hipError_t launch_experts(Epilogue e, const Product& p, hipStream_t) {
  ++launches;
  expect(p.M % kBigRows == 0, "whole blocks");
  const int64_t cols = e == kSwiglu ? 128 : 256;
  expect(p.M / kBigRows * ((p.N + cols - 1) / cols) <= kMaxGroups, "one launch");
  if (e == kSwiglu) expect(p.a_rows * p.lda <= 0x7fffffff, "gathered offsets");
  experts(e, p, kBigRows, p.M / kBigRows, false);
  return hipSuccess;
}
}  // namespace fp8

namespace moe {
int report_hip(hipError_t) { return MOE_ERR_HIP; }
int64_t align_scratch_ints(int64_t P, int32_t E) { return ((P + 255) / 256 + 1) * E; }
static void align(const int32_t* ids, int64_t P, int32_t E, int32_t bm, int32_t* sorted, int32_t* blocks, int32_t* n) {
  ++launches;
  const int64_t most = P + (P < E ? P : E) * (bm - 1);
  need(ids, 4 * P, "ids");
  need(sorted, 4 * most, "sorted");
  need(blocks, 4 * (most / bm), "blocks");
  need(n, 4, "count");
}
hipError_t launch_align(const int32_t* ids, int64_t P, int32_t E, int32_t, int32_t bm, int32_t* sorted,
                        int32_t* blocks, int32_t* n, hipStream_t) {
  align(ids, P, E, bm, sorted, blocks, n);
  return hipSuccess;
}
hipError_t launch_align_multi(const int32_t* ids, int64_t P, int32_t E, int32_t, int32_t bm, int32_t* sorted,
                              int32_t* blocks, int32_t* n, int32_t* scratch, hipStream_t) {
  align(ids, P, E, bm, sorted, blocks, n);
  need(scratch, 4 * align_scratch_ints(P, E), "scratch");
  return hipSuccess;
}
hipError_t launch_combine(const float* y, const float*, const int32_t* ids, const float* w, uint16_t* out,
                          int64_t T, int32_t H, int32_t k, int32_t, int32_t, hipStream_t) {
  ++launches;
  need(y, 4 * T * k * H, "y");
  need(ids, 4 * T * k, "ids");
  need(w, 4 * T * k, "weights");
  need(out, 2 * T * H, "out");
  return hipSuccess;
}
}  // namespace moe

namespace balance {
hipError_t launch_forward(const Sizes& z, const void* scores, const int32_t* ids, const uint8_t* mask,
                          const int32_t* offsets, float* loss, int32_t* counts, int32_t* tokens,
                          void* workspace, hipStream_t) {
  ++launches;
  need(scores, z.T * z.S * (z.type == MOE_TYPE_FP32 ? 4 : 2), "scores");
  need(ids, 4 * z.T * z.k, "ids");
  if (mask) need(mask, z.T, "mask");
  if (offsets) need(offsets, 4 * (z.B + 1), "offsets");
  need(loss, 4, "loss");
  need(counts, 4 * (int64_t)z.B * z.S, "counts");
  need(tokens, 4 * z.B, "tokens");
  if (alone(z)) return expect(groups(z.T) == 1, "one work-group"), hipSuccess;
  const Workspace w(z);
  const char* at = (const char*)workspace;
  need(at + w.sums, 8 * pieces(z) * z.S, "sums");
  need(at + w.counts, 4 * pieces(z) * (z.S + 1), "pieces' counts");
  need(at + w.parts, 8 * (int64_t)z.B * column_groups(z.S), "parts");
  expect(groups(z.T) * group_tokens(z.T) >= z.T, "work-groups cover the tokens");
  expect(group_tokens(z.T) <= kWaves * kMostTokens, "tokens of a wave");
  expect(groups(z.T) * 64 * kWaves < (1ll << 32), "a launch");
  return hipSuccess;
}
hipError_t launch_backward(const Sizes& z, const float* dloss, const void* scores, const int32_t* counts,
                           const int32_t* tokens, const uint8_t*, const int32_t*, void* dscores, hipStream_t) {
  ++launches;
  const int64_t n = z.T * z.S * (z.type == MOE_TYPE_FP32 ? 4 : 2);
  need(dloss, 4, "dloss");
  need(scores, n, "scores");
  need(dscores, n, "dscores");
  need(counts, 4 * (int64_t)z.B * z.S, "counts");
  need(tokens, 4 * z.B, "tokens");
  return hipSuccess;
}
}  // namespace balance

namespace {
void ok(int status, const char* what) {
  ++cases;
  if (status != MOE_OK) std::fprintf(stderr, "%s: status %d\n", what, status), ++failed;
}
int64_t sq(int64_t rows, int64_t width) { return 4 * fp8::blocks_of(rows) * fp8::blocks_of(width); }

void products(int64_t M, int32_t N, int32_t K) {
  for (int type : {MOE_TYPE_BF16, MOE_TYPE_FP32})
    for (int block : {1, 128})
      for (int quantize : {0, 1}) {
        buffers.clear();
        size_t n = 0;
        ok(moe_fp8_matmul_workspace_size(M, N, K, quantize, &n), "workspace");
        void* a = buffer((quantize ? 2 : 1) * M * K);
        float* as = quantize ? nullptr : (float*)buffer(row_scales(M, K));
        uint8_t* b = (uint8_t*)buffer((size_t)N * K);
        float* bs = (float*)buffer(block == 1 ? row_scales(N, K) : sq(N, K));
        void* out = buffer(M * N * (type == MOE_TYPE_BF16 ? 2 : 4));
        ok(moe_fp8_matmul(a, as, b, bs, block, M, N, K, type, out, buffer(n), n, nullptr), "matmul");
      }
  if (M > 1 << 20 || N > 1 << 20) return;
  for (int type : {MOE_TYPE_BF16, MOE_TYPE_FP32})
    for (int which : {1, 2, 3}) {
      buffers.clear();
      size_t n = 0;
      ok(moe_fp8_matmul_backward_workspace_size(M, N, K, &n), "workspace");
      const int size = type == MOE_TYPE_BF16 ? 2 : 4;
      void* dout = buffer(2 * M * N);
      void* a = which & 2 ? buffer(2 * M * K) : nullptr;
      uint8_t* b = which & 1 ? (uint8_t*)buffer((size_t)N * K) : nullptr;
      float* bs = which & 1 ? (float*)buffer(sq(N, K)) : nullptr;
      void* da = which & 1 ? buffer(size * M * K) : nullptr;
      void* db = which & 2 ? buffer((size_t)size * N * K) : nullptr;
      ok(moe_fp8_matmul_backward(dout, a, b, bs, M, N, K, type, da, db, buffer(n), n, nullptr), "backward");
    }
}
void experts(int64_t T, int32_t H, int32_t I, int32_t E, int32_t k) {
  buffers.clear();
  const moe_fp8_experts_problem p{T, H, I, E, 0, k};
  size_t n = 0;
  ok(moe_fp8_experts_workspace_size(&p, &n), "workspace");
  fp8::experts_of = E, fp8::tokens_of = T;
  void* x = buffer(2 * T * H);
  int32_t* ids = (int32_t*)buffer(4 * T * k);
  float* w = (float*)buffer(4 * T * k);
  uint8_t* w13 = (uint8_t*)buffer((size_t)E * 2 * I * H);
  float* s13 = (float*)buffer(E * sq(2 * I, H));
  uint8_t* w2 = (uint8_t*)buffer((size_t)E * I * H);
  float* s2 = (float*)buffer(E * sq(H, I));
  void* out = buffer(2 * T * H);
  ok(moe_fp8_experts_forward(x, ids, w, w13, s13, w2, s2, out, &p, buffer(n), n, nullptr), "experts");
}
void balances(int64_t T, int32_t S, int32_t k, int32_t B, int32_t type) {
  buffers.clear();
  const moe_balance_problem p{T, S, k, B, type};
  size_t n = 0;
  ok(moe_balance_workspace_size(&p, &n), "workspace");
  const size_t bytes = T * S * (type == MOE_TYPE_FP32 ? 4 : 2);
  void* scores = buffer(bytes);
  int32_t* ids = (int32_t*)buffer(4 * T * k);
  uint8_t* mask = (uint8_t*)buffer(T);
  int32_t* off = (int32_t*)buffer(4 * (B + 1));
  float* loss = (float*)buffer(4);
  int32_t* counts = (int32_t*)buffer(4 * (size_t)B * S);
  int32_t* tokens = (int32_t*)buffer(4 * B);
  ok(moe_balance_loss(scores, ids, mask, off, loss, counts, tokens, &p, buffer(n), n, nullptr), "balance");
  ok(moe_balance_loss_backward((float*)loss, scores, counts, tokens, mask, off, buffer(bytes), &p, nullptr),
     "balance gradient");
}
}  // namespace

int main() {
  for (int64_t M : {0, 1, 2, 4, 5, 16, 17, 33, 64, 65, 129, 777, 4096, 70001, 1 << 20})
    for (int32_t N : {8, 72, 1000, 4096, 100008})
      for (int32_t K : {16, 144, 1008, 7168, 14016, 1 << 20}) products(M, N, K);
  products(2314, 3456, 1232), products(5390, 2968, 1712), products(8783, 1800, 144);  // in two launches
  products((1ll << 31) - 256, 8, 16);
  products(8, 0x7fffff00, 16);
  for (int64_t M : {0, 1, 15, 127, 128, 129, 4099})
    for (int32_t K : {16, 128, 144, 7168})
      for (int type : {0, 1, 2})
        for (int block : {1, 128}) {
          buffers.clear();
          void* x = buffer(M * K * (type == 2 ? 4 : 2));
          uint8_t* c = (uint8_t*)buffer(M * K);
          float* s = (float*)buffer(block == 1 ? row_scales(M, K) : sq(M, K));
          ok(moe_fp8_quantize(x, type, M, K, block, c, s, nullptr), "quantize");
          ok(moe_fp8_dequantize(c, s, M, K, block, type, x, nullptr), "dequantize");
        }
  for (int64_t T : {0, 1, 2, 8, 63, 64, 200, 1024, 1025, 8191, 65536})
    for (int32_t H : {128, 384, 7168, 16384})
      for (int32_t E : {1, 7, 48, 512})
        for (int32_t k : {1, 8, 16}) experts(T, H, H == 384 ? 256 : 2048, E, k);
  for (int64_t T : {0ll, 1ll, 128ll, 129ll, 4096ll, 4097ll, 32768ll, 1000003ll, 1ll << 30})
    for (int32_t S : {1, 8, 65, 384, 1024})
      for (int32_t B : {1, 3, 8192})
        for (int type : {0, 1, 2}) balances(T, S, 1, B, type);
  std::printf("cases: %d launches: %d failed: %d\n", cases, launches, failed);
  return failed != 0;
}
