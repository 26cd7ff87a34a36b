// The host code of include/moe_ffn.h (csrc/ffn_api.cpp, csrc/ffn_plan.cpp) over
// many sizes, with the launches replaced by checks: every array a launch is
// handed lies, with the size the kernel addresses, in a buffer of the caller or
// in the workspace of exactly the size the library asked for; plans cover their
// product. No GPU.
#include <cstdio>
#include <vector>

#include "ffn_internal.h"
#include "moe_ffn.h"

namespace {
struct Buffer {
  const char* at;
  size_t bytes;
};
std::vector<Buffer> buffers;
int failed = 0, launches = 0, cases = 0;

void need(const void* p, size_t bytes, const char* what) {
  if (bytes == 0) return;
  const char* c = static_cast<const char*>(p);
  for (const Buffer& b : buffers)
    if (c >= b.at && c + bytes <= b.at + b.bytes) return;
  std::fprintf(stderr, "%s: %zu bytes at %p outside every buffer\n", what, bytes, p);
  ++failed;
}
void expect(bool ok, const char* what) {
  if (!ok) std::fprintf(stderr, "failed: %s\n", what), ++failed;
}

bool paired(ffn::Epilogue e) { return e == ffn::kSwiglu || e == ffn::kSwigluMx || e == ffn::kSwigluF32; }
void outputs(ffn::Epilogue e, const ffn::Product& p) {
  const size_t n = (size_t)p.M * p.N;
  switch (e) {
    case ffn::kStoreBf16: need(p.out, 2 * n, "out"); break;
    case ffn::kStoreF32: case ffn::kSwigluF32: need(p.out, 4 * n, "out"); break;
    case ffn::kSwiglu:
      need(p.out, 2 * n, "h");
      if (p.aux) need(p.aux, 8 * n, "gate_up");
      break;
    case ffn::kSwigluMx:
      need(p.out, n / 2, "h codes");
      need(p.aux, ffn::scale_bytes(p.M, p.N), "h scales");
      break;
    case ffn::kSwigluGrad:
      need(p.aux, 8 * n, "gate_up");
      need(p.out, 4 * n, "gradients of g and u");
      need(p.out2, 2 * n, "h");
      break;
    default: expect(false, "epilogue");
  }
}
void cut(const ffn::Cut& c, bool pair, int64_t M, int64_t N, int64_t K, bool mx) {
  const int64_t stages = (K + (mx ? 255 : 63)) / (mx ? 256 : 64);
  const int64_t tile_rows[] = {128, 128, 256, 64}, tile_cols[] = {128, 256, 256, 64};
  expect(c.tile >= 0 && c.tile <= 3, "tile");
  const int64_t rows = tile_rows[c.tile], cols = tile_cols[c.tile] / (pair ? 2 : 1);
  expect(c.groups == ((M + rows - 1) / rows) * ((N + cols - 1) / cols), "work-groups");
  expect(c.shares >= 1 && (c.tile == 0 || c.tile == 3 || c.shares == 1), "shares");
  if (c.tile == 0 || c.tile == 3) {
    expect((int64_t)c.share * c.shares >= stages, "the shares cover K");
    expect(c.shares == 1 || (int64_t)c.share * (c.shares - 1) < stages, "no empty share");
  }
}
}  // namespace

namespace ffn {
static void operands(Layout l, Epilogue e, const Product& p) {
  const size_t rows_b = (size_t)p.N * (paired(e) ? 2 : 1);
  if (l == kTN) {
    if (p.K) need(p.a, (p.K - 1) * p.lda + 2 * p.M, "a");
  } else {
    need(p.a, (p.M - 1) * p.lda + 2 * p.K, "a");
  }
  if (l == kNT)
    need(p.b, (rows_b - 1) * p.ldb + 2 * p.K, "b");
  else if (p.K)
    need(p.b, (p.K - 1) * p.ldb + 2 * p.N, "b");
  outputs(e, p);
}
hipError_t launch_product(Layout l, Epilogue e, const Product& p, void* split, hipStream_t) {
  ++launches;
  operands(l, e, p);
  need(split, product_workspace(l, e, p.M, p.N, p.K, false), "sums");
  return hipSuccess;
}
hipError_t launch_product_mx(Epilogue e, const Product& p, void* split, hipStream_t) {
  ++launches;
  const size_t rows_b = (size_t)p.N * (paired(e) ? 2 : 1);
  need(p.a, p.M * p.K / 2, "a");
  need(p.b, rows_b * p.K / 2, "b");
  need(p.a_scales, scale_bytes(p.M, p.K), "a scales");
  need(p.b_scales, scale_bytes(rows_b, p.K), "b scales");
  outputs(e, p);
  need(split, product_workspace(kNT, e, p.M, p.N, p.K, true), "sums");
  return hipSuccess;
}
hipError_t launch_gradients(const GradientsPlan& plan, const Product (&d)[3], void* split,
                            hipStream_t) {
  ++launches;
  expect(plan.together, "together");
  need(split, plan.bytes, "sums");
  size_t at = 0;
  for (int i = 0; i < 3; ++i) {
    operands(i ? kTN : kNN, kStoreBf16, d[i]);
    cut(plan.cut[i], false, d[i].M, d[i].N, d[i].K, false);
    if (plan.cut[i].shares == 1) continue;
    expect(plan.sums[i] == at && at % 16 == 0, "place of the sums");
    at += 4 * (size_t)d[i].M * d[i].N * plan.cut[i].shares;
  }
  expect(at == plan.bytes, "bytes of the sums");
  return hipSuccess;
}
hipError_t launch_rows(Epilogue e, const Product& p, hipStream_t) {
  ++launches;
  need(p.a, 2 * p.M * p.K, "a");
  need(p.b, (size_t)p.N * (paired(e) ? 2 : 1) * 2 * p.K, "b");
  outputs(e, p);
  expect(rows_fit(p, false, kAAsIs, paired(e)), "rows_fit");
  return hipSuccess;
}
hipError_t launch_rows_mx(Epilogue e, AType a, const Product& p, hipStream_t) {
  ++launches;
  const size_t rows_b = (size_t)p.N * (paired(e) ? 2 : 1);
  need(p.a, a == kAAsIs ? p.M * p.K / 2 : p.M * p.K * (a == kABf16 ? 2 : 4), "a");
  if (a == kAAsIs) need(p.a_scales, p.M * p.K / 32, "a scales");
  need(p.b, rows_b * p.K / 2, "b");
  need(p.b_scales, rows_b * p.K / 32, "b scales");
  outputs(e, p);
  expect(rows_fit(p, true, a, paired(e)), "rows_fit");
  return hipSuccess;
}
hipError_t launch_mx_quantize(const void* x, int32_t type, int64_t rows, int32_t width, uint8_t* codes,
                              uint8_t* scales, hipStream_t) {
  ++launches;
  need(x, rows * width * (type == MOE_TYPE_FP32 ? 4 : 2), "x");
  need(codes, rows * width / 2, "codes");
  need(scales, rows * (width / 32), "scales");
  return hipSuccess;
}
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t width,
                                int32_t type, void* out, hipStream_t) {
  ++launches;
  need(codes, rows * width / 2, "codes");
  need(scales, rows * (width / 32), "scales");
  need(out, rows * width * (type == MOE_TYPE_FP32 ? 4 : 2), "out");
  return hipSuccess;
}
hipError_t launch_mx_prepare(const void* x, int64_t rows, int32_t width, uint8_t* codes, uint8_t* scales,
                             const ScaleCopy& s0, const ScaleCopy& s1, hipStream_t) {
  ++launches;
  if (x) {
    need(x, 2 * rows * width, "x");
    need(codes, rows * width / 2, "codes");
    need(scales, scale_bytes(rows, width), "scales");
  }
  for (const ScaleCopy* s : {&s0, &s1})
    if (s->src) {
      need(s->src, s->rows * (s->width / 32), "given scales");
      need(s->dst, scale_bytes(s->rows, s->width), "scales by stage");
    }
  return hipSuccess;
}
}  // namespace ffn

namespace moe {
int report_hip(hipError_t) { return MOE_ERR_HIP; }
}  // namespace moe

namespace {
// callers' buffers at made-up addresses, 1 TiB apart; nothing reads them
char* fake(size_t bytes) {
  static char* next = reinterpret_cast<char*>(uintptr_t(1) << 44);
  char* p = next;
  next += size_t(1) << 40;
  buffers.push_back({p, bytes});
  return p;
}

void block(int64_t T, int32_t H, int32_t I) {
  ++cases;
  const moe_ffn_problem p{T, H, I};
  const bool mx = H % 32 == 0 && I % 32 == 0;
  for (int keep = 0; keep < 2; ++keep) {
    buffers.clear();
    size_t ws = 0;
    expect(moe_ffn_workspace_size(&p, MOE_FFN_FORWARD, &ws) == MOE_OK, "size");
    char *x = fake(2 * T * H), *w13 = fake(4ull * I * H), *w2 = fake(2ull * H * I), *o = fake(2 * T * H);
    char* gu = fake(8 * T * I);
    char* w = fake(ws);
    expect(moe_ffn_forward(x, w13, w2, o, keep ? (float*)gu : nullptr, &p, w, ws, nullptr) == MOE_OK,
           "forward");
    if (ws)
      expect(moe_ffn_forward(x, w13, w2, o, nullptr, &p, w, ws - 1, nullptr) == MOE_ERR_WORKSPACE,
             "forward, a byte short");
    buffers.clear();
    expect(moe_ffn_workspace_size(&p, MOE_FFN_BACKWARD, &ws) == MOE_OK, "size");
    x = fake(2 * T * H), w13 = fake(4ull * I * H), w2 = fake(2ull * H * I), gu = fake(8 * T * I);
    char *d = fake(2 * T * H), *dx = fake(2 * T * H), *d13 = fake(4ull * I * H), *d2 = fake(2ull * H * I);
    w = fake(ws);
    expect(moe_ffn_backward(d, x, (float*)gu, w13, w2, keep ? dx : nullptr, d13, d2, &p, w, ws,
                            nullptr) == MOE_OK, "backward");
  }
  if (!mx) return;
  buffers.clear();
  size_t ws = 0;
  expect(moe_ffn_workspace_size(&p, MOE_FFN_FORWARD_MXFP4, &ws) == MOE_OK, "size");
  const size_t n13 = 2ull * I * H, n2 = (size_t)H * I;
  char *x = fake(2 * T * H), *a = fake(n13 / 2), *sa = fake(n13 / 32), *b = fake(n2 / 2);
  char *sb = fake(n2 / 32), *o = fake(2 * T * H), *w = fake(ws);
  expect(moe_mxfp4_ffn_forward(x, (uint8_t*)a, (uint8_t*)sa, (uint8_t*)b, (uint8_t*)sb, o, &p, w, ws,
                               nullptr) == MOE_OK, "mxfp4 forward");
}

void product(int64_t M, int32_t N, int32_t K) {
  ++cases;
  for (int codes = 0; codes < 2; ++codes)
    for (int type : {MOE_TYPE_BF16, MOE_TYPE_FP32}) {
      buffers.clear();
      size_t ws = 0;
      expect(moe_mxfp4_matmul_workspace_size(M, N, K, !codes, &ws) == MOE_OK, "size");
      char *a = fake(codes ? M * K / 2 : 2 * M * K), *sa = fake(M * K / 32);
      char *b = fake((size_t)N * K / 2), *sb = fake((size_t)N * K / 32);
      char *o = fake((type == MOE_TYPE_FP32 ? 4 : 2) * M * N), *w = fake(ws);
      expect(moe_mxfp4_matmul(a, codes ? (uint8_t*)sa : nullptr, (uint8_t*)b, (uint8_t*)sb, M, N, K, type,
                              o, w, ws, nullptr) == MOE_OK, "matmul");
      if (ws)
        expect(moe_mxfp4_matmul(a, codes ? (uint8_t*)sa : nullptr, (uint8_t*)b, (uint8_t*)sb, M, N, K,
                                type, o, w, ws - 1, nullptr) == MOE_ERR_WORKSPACE, "a byte short");
    }
}

void plan(int64_t M, int64_t N, int64_t K) {
  ++cases;
  for (int mx = 0; mx < 2; ++mx)
    for (int l = 0; l < (mx ? 1 : 3); ++l)
      for (ffn::Epilogue e : {ffn::kStoreBf16, ffn::kSwiglu}) {
        const ffn::Plan p = ffn::plan_of(e, M, N, K, (ffn::Layout)l, mx);
        if (p.first) {
          expect(p.first % 256 == 0 && p.first < M, "first rows");
          expect(p.whole.tile == 2, "whole rounds of the large tile");
          cut(p.whole, e == ffn::kSwiglu, p.first, N, K, mx);
          cut(p.rest, e == ffn::kSwiglu, M - p.first, N, K, mx);
        } else {
          cut(p.whole, e == ffn::kSwiglu, M, N, K, mx);
        }
      }
}
}  // namespace

int main() {
  const int64_t rows[] = {0, 1, 2, 16, 17, 31, 64, 65, 130, 333, 1000, 4096, 4100, 70001, 2100003};
  const int32_t widths[][2] = {{8, 8}, {32, 32}, {64, 32}, {72, 40}, {696, 256}, {1000, 680}, {992, 736},
                               {7168, 256}, {7168, 2048}, {16640, 64}, {14336, 2112}, {1 << 20, 1 << 13}};
  for (int64_t T : rows)
    for (const auto& w : widths) block(T, w[0], w[1]);
  for (int64_t M : rows)
    for (int32_t N : {8, 72, 512, 4096, 4232, 40000})
      for (int32_t K : {32, 96, 544, 2048, 7168, 1 << 20}) product(M, N, K);
  for (int64_t M : {1, 16, 127, 128, 129, 700, 4096, 4100, 7168, 131072, 3000000})
    for (int64_t N : {8, 64, 200, 680, 2048, 2112, 7168, 100000})
      for (int64_t K : {0, 8, 64, 200, 2048, 7168, 1 << 20, 2000000}) plan(M, N, K);
  // the most rows, narrow enough to exist: every launch's lanes fit 32 bits
  const int64_t most = (int64_t(1) << 31) - 256;
  block(most, 8, 8);
  block(most, 32, 32);
  product(most, 8, 32);
  for (int64_t n : {8, 32, 64, 72})
    for (int64_t k : {8, 32, 64, 72})
      for (int mx = 0; mx < 2; ++mx)
        for (int l = 0; l < (mx ? 1 : 2); ++l)
          for (ffn::Epilogue e : {ffn::kStoreBf16, ffn::kSwiglu}) {
            const ffn::Plan p = ffn::plan_of(e, most, n, k, (ffn::Layout)l, mx);
            expect(p.whole.groups <= 0x7fffff && p.rest.groups <= 0x7fffff, "lanes of a launch");
          }
  std::printf("cases: %d launches: %d failed: %d\n", cases, launches, failed);
  return failed ? 1 : 0;
}
