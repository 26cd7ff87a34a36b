// The launches of a tiled product (each_launch, csrc/ffn_internal.h): row ranges
// that follow each other from the first row to the last, start at whole tiles of
// the cut and hold no more work-groups than a launch takes. No GPU.
#include <cstdio>

#include "ffn_internal.h"

namespace {
int failed = 0, cases = 0, split = 0;
void expect(bool ok, const char* what, int64_t M, int64_t N, int64_t K) {
  if (ok) return;
  std::fprintf(stderr, "%s: %lld x %lld x %lld\n", what, (long long)M, (long long)N, (long long)K);
  ++failed;
}
void product(ffn::Epilogue e, ffn::Layout l, int64_t M, int64_t N, int64_t K, bool mx) {
  ++cases;
  const ffn::Plan plan = ffn::plan_of(e, M, N, K, l, mx);
  const int64_t tile_rows[] = {128, 128, 256, 64}, tile_cols[] = {128, 256, 256, 64};
  const bool paired = e == ffn::kSwiglu || e == ffn::kSwigluMx;
  int64_t at = 0;
  int launches = 0;
  const hipError_t status =
      ffn::each_launch(plan, M, [&](int64_t first, int64_t end, const ffn::Cut& c) {
        const int64_t rows = tile_rows[c.tile], cols = tile_cols[c.tile] / (paired ? 2 : 1);
        const ffn::Cut& of = plan.first && first >= plan.first ? plan.rest : plan.whole;
        expect(first == at && first < end && end <= M, "rows in turn", M, N, K);
        expect((first - (&of == &plan.rest ? plan.first : 0)) % rows == 0 && first % 2 == 0,
               "whole tiles", M, N, K);
        expect(c.tile == of.tile && c.shares == of.shares && c.share == of.share, "cut", M, N, K);
        expect(c.groups == (end - first + rows - 1) / rows * ((N + cols - 1) / cols), "work-groups",
               M, N, K);
        expect(c.groups * (c.tile == 1 || c.tile == 2 ? 512 : 256) < (int64_t(1) << 32), "lanes",
               M, N, K);
        // sums are laid out for all rows of a cut: shares only where one launch has them
        expect(c.shares == 1 || c.groups == of.groups, "shares", M, N, K);
        at = end;
        ++launches;
        return hipSuccess;
      });
  expect(status == hipSuccess && at == M, "all rows", M, N, K);
  if (launches > (plan.first ? 2 : 1)) ++split;
  int calls = 0;
  const hipError_t stop = ffn::each_launch(plan, M, [&](int64_t, int64_t, const ffn::Cut&) {
    ++calls;
    return hipErrorInvalidValue;
  });
  expect(stop == hipErrorInvalidValue && calls == 1, "an error ends it", M, N, K);
}
}  // namespace

int main() {
  const int64_t most = (int64_t(1) << 31) - 256;
  for (int64_t M : {int64_t(1), int64_t(129), int64_t(4100), int64_t(70001), int64_t(1) << 30,
                    (int64_t(1) << 30) + 1, most})
    for (int64_t N : {int64_t(8), int64_t(160), int64_t(264), int64_t(7168), int64_t(1) << 20, most})
      for (int64_t K : {8, 32, 544, 7168})
        for (int mx = 0; mx < 2; ++mx)
          for (int l = 0; l < (mx ? 1 : 3); ++l)
            for (ffn::Epilogue e : {ffn::kStoreBf16, mx ? ffn::kSwigluMx : ffn::kSwiglu}) {
              if (e != ffn::kStoreBf16 && N > (1 << 20)) continue;
              if (M > (int64_t(1) << 42) / N) continue;  // results of 8 TB: millions of launches
              product(e, (ffn::Layout)l, M, N, K, mx);
            }
  // the MXFP4 block on 2^30 + 1 tokens at 32/160: 8388610 work-groups and 257 GB in all
  const int before = split;
  product(ffn::kSwigluMx, ffn::kNT, (int64_t(1) << 30) + 1, 160, 32, true);
  expect(split == before + 1, "more than one launch", (int64_t(1) << 30) + 1, 160, 32);
  std::printf("cases: %d in row ranges: %d failed: %d\n", cases, split, failed);
  return failed ? 1 : 0;
}
