// ffn_api.cpp -- host side of include/moe_ffn.h: argument checks, workspace
// layout and launch sequences. Every check runs before the first launch.
#include <algorithm>

#include "../../include/moe_ffn.h"
#include "ffn_internal.h"
#include "internal.h"

namespace {

using ffn::Product;

constexpr int32_t kMaxWidth = 1 << 20;
constexpr int64_t kMaxRows = 0x7fffff00;  // whole 256-row tiles below 2^31

size_t region(int64_t bytes) { return ((size_t)bytes + 255) / 256 * 256; }

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int check_problem(const moe_ffn_problem* p, int32_t multiple) {
  if (!p) return MOE_ERR_NULL;
  if (p->num_tokens < 0 || p->num_tokens > kMaxRows || p->hidden <= 0 || p->inter <= 0 ||
      p->hidden > kMaxWidth || p->inter > kMaxWidth || p->hidden % multiple ||
      p->inter % multiple)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

int check_rows(int64_t rows, int32_t width) {
  if (rows < 0 || rows > kMaxRows || width <= 0 || width > kMaxWidth || width % 32)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

// every pointer given, then every one aligned
int check_pointers(const void* const* ptrs, int n) {
  for (int i = 0; i < n; ++i)
    if (!ptrs[i]) return MOE_ERR_NULL;
  for (int i = 0; i < n; ++i)
    if (!aligned16(ptrs[i])) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return MOE_OK;
  if (!ws) return MOE_ERR_NULL;
  if (!aligned16(ws)) return MOE_ERR_ALIGNMENT;
  return have < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

int done(hipError_t e) { return e == hipSuccess ? MOE_OK : moe::report_hip(e); }

// MXFP4 [rows, width] in a workspace: codes, then scales by stage
struct MxRegion {
  size_t codes, scales;
  MxRegion(int64_t rows, int32_t width)
      : codes(region(rows * (width / 2))), scales(region(ffn::scale_bytes(rows, width))) {}
  size_t bytes() const { return codes + scales; }
};

// How a forward pass runs its products: tiled, or as the few-row kernels take
// them; in MXFP4 these quantise A themselves, or find x quantised by a launch
// ahead (more than 16 rows). The tiled estimate is that of its products; with it
// go what the launches' order costs and, in MXFP4, the launch that brings scales
// into the order of the stages (kAhead*, measured at 20 to 64 rows; the few-row
// kernels of codes have no launch ahead at all).
constexpr double kAheadBf16 = 2.0, kAheadMx = 4.5, kAheadCodes = 6.0;
enum Path { kTiled, kFew, kFewPrepared };

Path path_of(const moe_ffn_problem* p, bool mx) {
  Product up{}, down{};
  up.M = down.M = p->num_tokens;
  up.N = down.K = p->inter;
  up.K = down.N = p->hidden;
  if (!ffn::rows_fit(down, mx, mx ? ffn::kAF32 : ffn::kAAsIs, false)) return kTiled;
  Path few = kFew;
  if (!ffn::rows_fit(up, mx, mx ? ffn::kABf16 : ffn::kAAsIs, true)) {
    if (!mx || !ffn::rows_fit(up, mx, ffn::kAAsIs, true)) return kTiled;
    few = kFewPrepared;
  }
  if (p->num_tokens <= 16 && few == kFew) return few;
  const ffn::Epilogue swiglu = mx ? ffn::kSwigluMx : ffn::kSwiglu;
  const double tiled =
      ffn::product_time(ffn::kNT, swiglu, up.M, up.N, up.K, mx) +
      ffn::product_time(ffn::kNT, ffn::kStoreBf16, down.M, down.N, down.K, mx);
  const double rows = ffn::rows_time(up, mx, ffn::kAAsIs, true) +
                      ffn::rows_time(down, mx, mx ? ffn::kAF32 : ffn::kAAsIs, false);
  return rows < tiled + (mx ? kAheadMx : kAheadBf16) ? few : kTiled;
}

Path path_of(int64_t rows, int32_t cols, int32_t width, bool quantize) {
  Product d{};
  d.M = rows, d.N = cols, d.K = width;
  if (ffn::rows_fit(d, true, quantize ? ffn::kABf16 : ffn::kAAsIs, false) && rows <= 16)
    return kFew;
  if (!ffn::rows_fit(d, true, ffn::kAAsIs, false)) return kTiled;
  const double tiled = ffn::product_time(ffn::kNT, ffn::kStoreF32, rows, cols, width, true);
  return ffn::rows_time(d, true, ffn::kAAsIs, false) < tiled + (quantize ? kAheadMx : kAheadCodes)
             ? quantize ? kFewPrepared : kFew
             : kTiled;
}

// x in MXFP4 as the few-row kernels read it: codes, then K/32 bytes a row
struct RowRegion {
  size_t codes, scales;
  RowRegion(int64_t rows, int32_t width)
      : codes(region(rows * (width / 2))), scales(region(rows * (width / 32))) {}
  size_t bytes() const { return codes + scales; }
};

// The shares' sums of a pass's products, which follow each other: one region
size_t split_of(const moe_ffn_problem* p, int pass) {
  const int64_t T = p->num_tokens, H = p->hidden, I = p->inter;
  const bool mx = pass == MOE_FFN_FORWARD_MXFP4;
  size_t most = 0;
  auto add = [&](ffn::Layout layout, ffn::Epilogue epi, int64_t M, int64_t N, int64_t K) {
    most = std::max(most, ffn::product_workspace(layout, epi, M, (int32_t)N, K, mx));
  };
  if (pass == MOE_FFN_BACKWARD) {
    add(ffn::kNN, ffn::kSwigluGrad, T, I, H);
    add(ffn::kNN, ffn::kStoreBf16, T, H, 2 * I);
    add(ffn::kTN, ffn::kStoreBf16, 2 * I, H, T);
    add(ffn::kTN, ffn::kStoreBf16, H, I, T);
    most = std::max(most, ffn::gradients_plan(T, H, I).bytes);
  } else {
    add(ffn::kNT, mx ? ffn::kSwigluMx : ffn::kSwiglu, T, I, H);
    add(ffn::kNT, ffn::kStoreBf16, T, H, I);
  }
  return region(most);
}

size_t workspace_of(const moe_ffn_problem* p, int pass) {
  const int64_t T = p->num_tokens, H = p->hidden, I = p->inter;
  if (T == 0) return 0;
  if (pass == MOE_FFN_BACKWARD)
    return region(4 * T * I) + region(2 * T * I) + split_of(p, pass);
  if (pass == MOE_FFN_FORWARD)
    return region(2 * T * I) + (path_of(p, false) == kTiled ? split_of(p, pass) : 0);
  const Path path = path_of(p, true);
  if (path != kTiled)
    return region(4 * T * I) + (path == kFewPrepared ? RowRegion(T, p->hidden).bytes() : 0);
  return MxRegion(T, p->hidden).bytes() + MxRegion(T, p->inter).bytes() +
         region(ffn::scale_bytes(2 * I, H)) + region(ffn::scale_bytes(H, I)) + split_of(p, pass);
}

}  // namespace

extern "C" {

int moe_ffn_workspace_size(const moe_ffn_problem* p, int pass, size_t* bytes) {
  if (!p || !bytes) return MOE_ERR_NULL;
  if (pass < MOE_FFN_FORWARD || pass > MOE_FFN_FORWARD_MXFP4) return MOE_ERR_UNSUPPORTED;
  const int st = check_problem(p, pass == MOE_FFN_FORWARD_MXFP4 ? 32 : 8);
  if (st != MOE_OK) return st;
  *bytes = workspace_of(p, pass);
  return MOE_OK;
}

int moe_ffn_forward(const void* x, const void* w13, const void* w2, void* out, float* gate_up,
                    const moe_ffn_problem* p, void* workspace, size_t workspace_bytes,
                    void* stream) {
  int st = check_problem(p, 8);
  if (st != MOE_OK || p->num_tokens == 0) return st;
  const void* ptrs[] = {x, w13, w2, out};
  if ((st = check_pointers(ptrs, 4)) != MOE_OK) return st;
  if (gate_up && !aligned16(gate_up)) return MOE_ERR_ALIGNMENT;
  st = check_workspace(workspace, workspace_bytes, workspace_of(p, MOE_FFN_FORWARD));
  if (st != MOE_OK) return st;
  const int64_t T = p->num_tokens, H = p->hidden, I = p->inter;
  hipStream_t s = (hipStream_t)stream;
  Product up{x, w13, nullptr, nullptr, 2 * H, 2 * H, T, p->inter, H};
  up.out = workspace;
  up.aux = gate_up;
  Product down{workspace, w2, nullptr, nullptr, 2 * I, 2 * I, T, p->hidden, I};
  down.out = out;
  const bool few = path_of(p, false) != kTiled;
  char* split = (char*)workspace + region(2 * T * I);
  const hipError_t e = few ? ffn::launch_rows(ffn::kSwiglu, up, s)
                           : ffn::launch_product(ffn::kNT, ffn::kSwiglu, up, split, s);
  if (e != hipSuccess) return done(e);
  return done(few ? ffn::launch_rows(ffn::kStoreBf16, down, s)
                  : ffn::launch_product(ffn::kNT, ffn::kStoreBf16, down, split, s));
}

int moe_ffn_backward(const void* dout, const void* x, const float* gate_up, const void* w13,
                     const void* w2, void* dx, void* dw13, void* dw2, const moe_ffn_problem* p,
                     void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_problem(p, 8);
  if (st != MOE_OK) return st;
  if (!dw13 != !dw2 || (!dx && !dw13)) return MOE_ERR_NULL;
  if (!aligned16(dx) || !aligned16(dw13) || !aligned16(dw2)) return MOE_ERR_ALIGNMENT;
  const int64_t T = p->num_tokens, H = p->hidden, I = p->inter;
  if (T > 0) {
    const void* ptrs[] = {dout, x, gate_up, w13, w2};
    if ((st = check_pointers(ptrs, 5)) != MOE_OK) return st;
    st = check_workspace(workspace, workspace_bytes, workspace_of(p, MOE_FFN_BACKWARD));
    if (st != MOE_OK) return st;
  }
  hipStream_t s = (hipStream_t)stream;
  char* dgu = (char*)workspace;                      // bf16 [T, 2I]
  char* h = T > 0 ? dgu + region(4 * T * I) : dgu;   // bf16 [T, I]
  char* split = T > 0 ? h + region(2 * T * I) : dgu;
  hipError_t e = hipSuccess;
  if (T > 0) {
    Product dh{dout, w2, nullptr, nullptr, 2 * H, 2 * I, T, p->inter, H};
    dh.out = dgu;
    dh.out2 = h;
    dh.aux = const_cast<float*>(gate_up);
    e = ffn::launch_product(ffn::kNN, ffn::kSwigluGrad, dh, split, s);
  }
  Product d[3] = {{dgu, w13, nullptr, nullptr, 4 * I, 2 * H, T, p->hidden, 2 * I},
                  {dgu, x, nullptr, nullptr, 4 * I, 2 * H, 2 * I, p->hidden, T},
                  {dout, h, nullptr, nullptr, 2 * H, 2 * I, H, p->inter, T}};
  d[0].out = dx;
  d[1].out = dw13;
  d[2].out = dw2;
  if (e == hipSuccess && dx && dw13) {
    const ffn::GradientsPlan plan = ffn::gradients_plan(T, H, I);
    if (plan.together) return done(ffn::launch_gradients(plan, d, split, s));
  }
  if (e == hipSuccess && dx && T > 0)
    e = ffn::launch_product(ffn::kNN, ffn::kStoreBf16, d[0], split, s);
  for (int i = 1; i < 3 && e == hipSuccess && dw13; ++i)
    e = ffn::launch_product(ffn::kTN, ffn::kStoreBf16, d[i], split, s);
  return done(e);
}

int moe_mxfp4_quantize(const void* x, int32_t type, int64_t rows, int32_t width, uint8_t* codes,
                       uint8_t* scales, void* stream) {
  int st = check_rows(rows, width);
  if (st != MOE_OK) return st;
  if (type < MOE_TYPE_BF16 || type > MOE_TYPE_FP32) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const void* ptrs[] = {x, codes};
  if (!scales) return MOE_ERR_NULL;
  if ((st = check_pointers(ptrs, 2)) != MOE_OK) return st;
  return done(
      ffn::launch_mx_quantize(x, type, rows, width, codes, scales, (hipStream_t)stream));
}

int moe_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t width,
                         int32_t type, void* out, void* stream) {
  int st = check_rows(rows, width);
  if (st != MOE_OK) return st;
  if (type < MOE_TYPE_BF16 || type > MOE_TYPE_FP32) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const void* ptrs[] = {codes, out};
  if (!scales) return MOE_ERR_NULL;
  if ((st = check_pointers(ptrs, 2)) != MOE_OK) return st;
  return done(
      ffn::launch_mx_dequantize(codes, scales, rows, width, type, out, (hipStream_t)stream));
}

int moe_mxfp4_matmul_workspace_size(int64_t rows, int32_t cols, int32_t width, int quantize,
                                    size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const int st = check_rows(rows, width);
  if (st != MOE_OK) return st;
  if (cols <= 0 || cols > kMaxRows || cols % 8) return MOE_ERR_SHAPE;
  *bytes = 0;
  const Path path = rows == 0 ? kFew : path_of(rows, cols, width, quantize);
  if (path == kFewPrepared) *bytes = RowRegion(rows, width).bytes();
  if (path != kTiled) return MOE_OK;
  *bytes = (quantize ? MxRegion(rows, width).bytes() : region(ffn::scale_bytes(rows, width))) +
           region(ffn::scale_bytes(cols, width)) +
           region(ffn::product_workspace(ffn::kNT, ffn::kStoreF32, rows, cols, width, true));
  return MOE_OK;
}

int moe_mxfp4_matmul(const void* a, const uint8_t* a_scales, const uint8_t* b,
                     const uint8_t* b_scales, int64_t rows, int32_t cols, int32_t width,
                     int32_t out_type, void* out, void* workspace, size_t workspace_bytes,
                     void* stream) {
  size_t need = 0;
  int st = moe_mxfp4_matmul_workspace_size(rows, cols, width, !a_scales, &need);
  if (st != MOE_OK) return st;
  if (out_type != MOE_TYPE_BF16 && out_type != MOE_TYPE_FP32) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const void* ptrs[] = {a, b, out};
  if (!b_scales) return MOE_ERR_NULL;
  if ((st = check_pointers(ptrs, 3)) != MOE_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MOE_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  const ffn::Epilogue store = out_type == MOE_TYPE_FP32 ? ffn::kStoreF32 : ffn::kStoreBf16;
  const Path path = path_of(rows, cols, width, !a_scales);
  if (path != kTiled) {
    if (path == kFewPrepared) {
      uint8_t* codes = (uint8_t*)workspace;
      uint8_t* scales = codes + RowRegion(rows, width).codes;
      const hipError_t e =
          ffn::launch_mx_quantize(a, MOE_TYPE_BF16, rows, width, codes, scales, s);
      if (e != hipSuccess) return done(e);
      a = codes;
      a_scales = scales;
    }
    Product d{a, b, a_scales, b_scales, width / 2, width / 2, rows, cols, width};
    d.out = out;
    return done(ffn::launch_rows_mx(store, a_scales ? ffn::kAAsIs : ffn::kABf16, d, s));
  }
  uint8_t* sb = (uint8_t*)workspace;
  uint8_t* sa = sb + region(ffn::scale_bytes(cols, width));
  uint8_t* codes = sa + region(ffn::scale_bytes(rows, width));
  uint8_t* split = a_scales ? codes : codes + MxRegion(rows, width).codes;
  const ffn::ScaleCopy copy_b{b_scales, sb, cols, width};
  hipError_t e;
  if (a_scales) {
    e = ffn::launch_mx_prepare(nullptr, 0, 0, nullptr, nullptr, copy_b, {a_scales, sa, rows, width},
                               s);
  } else {
    e = ffn::launch_mx_prepare(a, rows, width, codes, sa, copy_b, {}, s);
    a = codes;
  }
  if (e != hipSuccess) return done(e);
  Product d{a, b, sa, sb, width / 2, width / 2, rows, cols, width};
  d.out = out;
  return done(ffn::launch_product_mx(store, d, split, s));
}

int moe_mxfp4_ffn_forward(const void* x, const uint8_t* w13, const uint8_t* w13_scales,
                          const uint8_t* w2, const uint8_t* w2_scales, void* out,
                          const moe_ffn_problem* p, void* workspace, size_t workspace_bytes,
                          void* stream) {
  int st = check_problem(p, 32);
  if (st != MOE_OK || p->num_tokens == 0) return st;
  const void* ptrs[] = {x, w13, w2, out};
  if (!w13_scales || !w2_scales) return MOE_ERR_NULL;
  if ((st = check_pointers(ptrs, 4)) != MOE_OK) return st;
  st = check_workspace(workspace, workspace_bytes, workspace_of(p, MOE_FFN_FORWARD_MXFP4));
  if (st != MOE_OK) return st;
  const int64_t T = p->num_tokens;
  const int32_t H = p->hidden, I = p->inter;
  hipStream_t s = (hipStream_t)stream;
  const Path path = path_of(p, true);
  if (path != kTiled) {
    Product up{x, w13, nullptr, w13_scales, H / 2, H / 2, T, I, H};
    up.out = workspace;
    hipError_t e = hipSuccess;
    if (path == kFewPrepared) {
      uint8_t* codes = (uint8_t*)workspace + region(4 * T * I);
      uint8_t* scales = codes + RowRegion(T, H).codes;
      e = ffn::launch_mx_quantize(x, MOE_TYPE_BF16, T, H, codes, scales, s);
      up.a = codes;
      up.a_scales = scales;
    }
    if (e == hipSuccess)
      e = ffn::launch_rows_mx(ffn::kSwigluF32, path == kFew ? ffn::kABf16 : ffn::kAAsIs, up, s);
    if (e != hipSuccess) return done(e);
    Product down{workspace, w2, nullptr, w2_scales, I / 2, I / 2, T, H, I};
    down.out = out;
    return done(ffn::launch_rows_mx(ffn::kStoreBf16, ffn::kAF32, down, s));
  }
  const MxRegion rx(T, H), rh(T, I);
  uint8_t* xc = (uint8_t*)workspace;
  uint8_t* xs = xc + rx.codes;
  uint8_t* hc = xc + rx.bytes();
  uint8_t* hs = hc + rh.codes;
  uint8_t* s13 = hc + rh.bytes();
  uint8_t* s2 = s13 + region(ffn::scale_bytes(2 * (int64_t)I, H));
  uint8_t* split = s2 + region(ffn::scale_bytes(H, I));
  hipError_t e = ffn::launch_mx_prepare(x, T, H, xc, xs, {w13_scales, s13, 2 * (int64_t)I, H},
                                        {w2_scales, s2, H, I}, s);
  if (e != hipSuccess) return done(e);
  Product up{xc, w13, xs, s13, H / 2, H / 2, T, I, H};
  up.out = hc;
  up.aux = hs;
  e = ffn::launch_product_mx(ffn::kSwigluMx, up, split, s);
  if (e != hipSuccess) return done(e);
  Product down{hc, w2, hs, s2, I / 2, I / 2, T, H, I};
  down.out = out;
  return done(ffn::launch_product_mx(ffn::kStoreBf16, down, split, s));
}

}  // extern "C"
