// Which kernels the host code of include/moe_fp8.h launches for a few rows, by the library's own rules
// (csrc/fp8_api.cpp, csrc/fp8_plan.cpp, csrc/fp8_rows_plan.cpp), the launches replaced by checks: every array
// a launch is handed lies in a buffer of the caller or in the workspace of exactly the size asked for,
// and a few-row launch fits the LDS of a CU. Lines on stdin, one line on stdout for each:
//
//   m M N K quantize block type   the launches of moe_fp8_matmul: q (quantise), r (few rows of codes),
//                                 f (few rows, quantised on the way), t (tiles)
//   e T H I E k                   moe_fp8_experts_forward: "few" and the slices of a work-group of both products,
//                                 or "tiles"
//   f source M N K                rows_fit
//   s tm tn                       experts_span
#include <cstdio>
#include <string>
#include <vector>

#include "fp8_internal.h"
#include "internal.h"
#include "moe_fp8.h"

namespace {
struct Buffer {
  const char* at;
  size_t bytes;
};
std::vector<Buffer> buffers;
std::string launched;
int failed = 0;
char* next_address = (char*)0x100000000000;
constexpr int64_t kLds = 160 * 1024;

// an address range of its own; nothing of it is touched
void* buffer(size_t bytes) {
  char* at = next_address;
  next_address += (bytes + 4096) / 4096 * 4096 + 4096;
  buffers.push_back({at, bytes});
  return at;
}
void need(const void* p, int64_t bytes, const char* what) {
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
int64_t square_scales(int64_t rows, int64_t width) {
  return 4 * fp8::blocks_of(rows) * fp8::blocks_of(width);
}
}  // namespace

namespace fp8 {
hipError_t launch_quantize(const void* x, int32_t, int64_t rows, int32_t width, int32_t,
                           uint8_t* codes, float* scales, hipStream_t) {
  launched += 'q';
  need(x, 2 * rows * width, "x");
  need(codes, rows * width, "codes");
  need(scales, row_scales(rows, width), "scales");
  return hipSuccess;
}
hipError_t launch_dequantize(const uint8_t*, const float*, int64_t, int32_t, int32_t, int32_t, void*, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_prepare(const Prepare&, hipStream_t) { return hipSuccess; }
hipError_t launch_clear(void*, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_product(Mode mode, Epilogue e, const Product& p, void* split, hipStream_t) {
  launched += 't';
  need(p.a, p.M * p.K, "a");
  need(p.a_scales, row_scales(p.M, p.K), "a's scales");
  const size_t sums = product_workspace(e == kStoreF32, mode == kRowScales, p.M, p.N, p.K);
  if (sums) need(split, sums, "sums");
  return hipSuccess;
}
hipError_t launch_rows(Source source, Epilogue e, const Product& p, hipStream_t) {
  launched += source == kCodes ? 'r' : 'f';
  expect(rows_fit(source, p.M, p.N, p.K), "few rows");
  expect(rows_extra(source != kCodes, p.M, p.K, 1) + kRowsStages * kRowsWaves * kRowsSlot <= kLds, "LDS");
  // B by 31-bit offsets from its first byte, the columns past its last row too
  expect(p.N * p.K <= 0x7fffffff, "offsets");
  need(p.a, (source == kCodes ? 1 : 2) * p.M * p.K, "a");
  if (source == kCodes) need(p.a_scales, row_scales(p.M, p.K), "a's scales");
  need(p.b, (int64_t)p.N * p.K, "b");
  need(p.b_scales, square_scales(p.N, p.K), "b's scales");
  need(p.out, p.M * p.N * (e == kStoreBf16 ? 2 : 4), "out");
  return hipSuccess;
}
hipError_t launch_experts_rows(Epilogue e, const Product& p, int64_t buckets, hipStream_t) {
  const int slices = experts_slices(e, p.N, p.K, buckets);
  launched += (launched.empty() ? "few " : " ") + std::to_string(slices);
  const int64_t extra = rows_extra(true, kFewRows, p.K, slices);
  // (the three stages that the ring does not have are 16 bytes each, 1 KB apart)
  expect(extra <= 64 * 1024 && extra + kExpertsStages * (kRowsWaves * kRowsSlot + 1024) <= kLds, "LDS");
  const int64_t across = (p.N + rows_step(e) - 1) / rows_step(e);
  expect(across % slices == 0 && 128 % (slices * rows_step(e)) == 0, "a work-group's columns in one block");
  expect((e == kSwiglu ? 2 : 1) * (int64_t)p.N * p.K <= 0x7fffffff, "offsets");
  return hipSuccess;
}
hipError_t launch_experts(Epilogue, const Product&, hipStream_t) {
  launched = "tiles";
  return hipSuccess;
}
}  // namespace fp8

namespace moe {
int report_hip(hipError_t) { return MOE_ERR_HIP; }
int64_t align_scratch_ints(int64_t P, int32_t E) { return ((P + 255) / 256 + 1) * E; }
hipError_t launch_align(const int32_t*, int64_t, int32_t, int32_t, int32_t, int32_t*, int32_t*, int32_t*,
                        hipStream_t) {
  launched.clear();
  return hipSuccess;
}
hipError_t launch_align_multi(const int32_t*, int64_t, int32_t, int32_t, int32_t, int32_t*, int32_t*, int32_t*,
                              int32_t*, hipStream_t) {
  launched.clear();
  return hipSuccess;
}
hipError_t launch_combine(const float*, const float*, const int32_t*, const float*, uint16_t*, int64_t, int32_t,
                          int32_t, int32_t, int32_t, hipStream_t) {
  return hipSuccess;
}
}  // namespace moe

int main() {
  char op;
  long long v[6];
  while (std::scanf(" %c", &op) == 1) {
    const int n = op == 'm' ? 6 : op == 'e' ? 5 : op == 's' ? 2 : 4;
    for (int i = 0; i < n; ++i)
      if (std::scanf("%lld", &v[i]) != 1) return 2;
    buffers.clear();
    launched.clear();
    size_t bytes = 0;
    if (op == 'm') {
      const int64_t M = v[0], N = v[1], K = v[2];
      const bool quantize = v[3] != 0, square = v[4] == 128;
      const int type = (int)v[5];
      expect(moe_fp8_matmul_workspace_size(M, N, K, quantize, &bytes) == MOE_OK, "workspace");
      void* a = buffer((quantize ? 2 : 1) * M * K);
      float* as = quantize ? nullptr : (float*)buffer(row_scales(M, K));
      uint8_t* b = (uint8_t*)buffer(N * K);
      float* bs = (float*)buffer(square ? square_scales(N, K) : row_scales(N, K));
      void* out = buffer(M * N * (type == MOE_TYPE_BF16 ? 2 : 4));
      expect(moe_fp8_matmul(a, as, b, bs, (int)v[4], M, N, K, type, out, buffer(bytes), bytes, nullptr) == MOE_OK,
             "matmul");
    } else if (op == 'e') {
      const int64_t T = v[0], H = v[1], I = v[2], E = v[3], k = v[4];
      const moe_fp8_experts_problem p{T, (int)H, (int)I, (int)E, 0, (int)k};
      expect(moe_fp8_experts_workspace_size(&p, &bytes) == MOE_OK, "workspace");
      void* x = buffer(2 * T * H);
      int32_t* ids = (int32_t*)buffer(4 * T * k);
      float* w = (float*)buffer(4 * T * k);
      uint8_t *w13 = (uint8_t*)buffer(E * 2 * I * H), *w2 = (uint8_t*)buffer(E * I * H);
      float *s13 = (float*)buffer(E * square_scales(2 * I, H)), *s2 = (float*)buffer(E * square_scales(H, I));
      expect(moe_fp8_experts_forward(x, ids, w, w13, s13, w2, s2, buffer(2 * T * H), &p, buffer(bytes), bytes,
                                     nullptr) == MOE_OK, "experts");
    } else if (op == 's') {
      launched = std::to_string(fp8::experts_span(v[0], v[1]));
    } else {
      launched = fp8::rows_fit((fp8::Source)v[0], v[1], v[2], v[3]) ? "1" : "0";
    }
    std::printf("%s\n", launched.c_str());
  }
  return failed != 0;
}
