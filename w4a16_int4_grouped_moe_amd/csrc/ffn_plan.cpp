// ffn_plan.cpp -- which kernel computes a product, and in which pieces: host
// arithmetic on the sizes, by times measured on the MI355X.
#include <algorithm>

#include "ffn_internal.h"

namespace ffn {
namespace {

constexpr int kMaxRows = 64;       // of the few-row kernels
constexpr int kMxLds = 64 * 1024;  // an A quantised in LDS, codes and scales

// Microseconds a stage of K takes one round of work-groups on 256 CUs, and what
// a work-group costs besides. Measured on products of 20 to 4096 rows at
// widths 256 to 7168 (bf16 with K contiguous operands; with a row contiguous
// one; MXFP4).
struct Rate {
  double stage[4], fixed[4];
};
constexpr Rate kRates[3] = {{{0.62, 0.88, 1.42, 0.32}, {4.5, 4.5, 7.0, 4.5}},
                            {{0.70, 0.85, 1.42, 0.36}, {4.0, 5.0, 7.0, 4.5}},
                            {{0.85, 1.20, 1.80, 0.40}, {4.5, 4.5, 8.0, 4.5}}};
// The cheapest cut. Shares of K cost a launch and the sums' way to memory and
// back (about 4 TB/s); of equals the larger tile.
Cut cut_of(Epilogue epi, int64_t M, int64_t N, int64_t K, Layout layout, bool mx) {
  const bool paired = epi == kSwiglu || epi == kSwigluMx;
  const Rate& rate = kRates[mx ? 2 : layout == kNT ? 0 : 1];
  const int64_t stages = (K + (mx ? 255 : 63)) / (mx ? 256 : 64);
  auto tiles = [&](int64_t rows, int64_t cols) {
    if (paired) cols /= 2;
    return ((M + rows - 1) / rows) * ((N + cols - 1) / cols);
  };
  auto time = [&](int tile, int64_t groups, int64_t st) {
    return (double)((groups + 255) / 256) * (st * rate.stage[tile] + rate.fixed[tile]);
  };
  // a tile's pre-activations on their way, which the join of shares reads at full rate
  const double grad = epi == kSwigluGrad ? 4.0 : 0.0;
  const int64_t n[4] = {tiles(128, 128), tiles(128, 256), tiles(256, 256), tiles(64, 64)};
  Cut best{2, 1, (int)stages, n[2]};
  double least = time(2, n[2], stages) + grad;
  if (time(1, n[1], stages) + grad < least) {
    least = time(1, n[1], stages) + grad;
    best = Cut{1, 1, (int)stages, n[1]};
  }
  for (int tile : {0, 3})
    for (int shares = 1; shares <= 32 && n[tile] * shares <= 1024; ++shares) {
      const int64_t share = (stages + shares - 1) / shares;
      if (shares > 1 && (2 * shares > stages || share * (shares - 1) >= stages)) continue;
      const double sums = 4.0 * M * N * (paired ? 2 : 1) * shares;
      const double t =
          time(tile, n[tile] * shares, share) + (shares > 1 ? 3.0 + 2 * sums / 4e6 : grad);
      if (t < least) least = t, best = Cut{tile, shares, (int)share, n[tile]};
    }
  best.time = least;
  return best;
}

}  // namespace

// A product whose last round of tiles is nearly empty is computed in two
// launches: its first rows in whole rounds of 256 x 256 tiles, the rest cut on
// its own (4100 tokens at 7168/2048: one round and 4 rows instead of two).
Plan plan_of(Epilogue epi, int64_t M, int64_t N, int64_t K, Layout layout, bool mx) {
  Plan best;
  best.whole = cut_of(epi, M, N, K, layout, mx);
  best.time = best.whole.time;
  const bool paired = epi == kSwiglu || epi == kSwigluMx;
  const int64_t cols = paired ? 128 : 256, tn = (N + cols - 1) / cols;
  const int64_t rounds = ((M + 255) / 256 * tn + 255) / 256;
  if (rounds < 2) return best;
  const int64_t rows = (rounds - 1) * 256 / tn * 256;  // of whole rounds
  if (rows <= 0 || rows >= M) return best;
  const Cut rest = cut_of(epi, M - rows, N, K, layout, mx);
  Cut first{2, 1, 0, rows / 256 * tn};
  const int64_t stages = (K + (mx ? 255 : 63)) / (mx ? 256 : 64);
  const Rate& rate = kRates[mx ? 2 : layout == kNT ? 0 : 1];
  first.time = (double)((first.groups + 255) / 256) * (stages * rate.stage[2] + rate.fixed[2]);
  if (first.time + rest.time + 3.0 < 0.95 * best.time)
    best.first = rows, best.whole = first, best.rest = rest,
    best.time = first.time + rest.time + 3.0;
  return best;
}

size_t product_workspace(Layout layout, Epilogue epilogue, int64_t M, int32_t N, int64_t K,
                         bool mx) {
  if (M == 0) return 0;
  const Plan plan = plan_of(epilogue, M, N, K, layout, mx);
  const bool paired = epilogue == kSwiglu || epilogue == kSwigluMx;
  const Cut& c = plan.first ? plan.rest : plan.whole;
  return c.shares > 1 ? (size_t)c.shares * (M - plan.first) * N * (paired ? 8 : 4) : 0;
}

double product_time(Layout layout, Epilogue epilogue, int64_t M, int32_t N, int64_t K, bool mx) {
  return plan_of(epilogue, M, N, K, layout, mx).time;
}

// All three shares of K are cut to about one length. In one launch no product
// waits for another: a round is as long as the longest share, more rounds are
// the CUs' parts of all the work and about half a share with some CUs idle.
// Whole backward pass, three launches -> one of 128 x 128 tiles (microseconds):
// 201 tokens at 1000/680 42 -> 29, 1000 at 1000/680 64 -> 38, 2000 at 512/128 46 ->
// 28, 700 at 2048/768 62 -> 42, 8192 at 512/512 82 -> 71, 4096 at 2048/256 77 either
// way. 64 x 64 against 128 x 128 tiles, replayed from a graph: 20 tokens at 696/256
// 13.4 and 16.9, 300 at 296/200 14.3 and 17.1.
GradientsPlan gradients_plan(int64_t tokens, int64_t hidden, int64_t inter) {
  const int64_t sizes[3][3] = {{tokens, hidden, 2 * inter},
                               {2 * inter, hidden, tokens},
                               {hidden, inter, tokens}};  // M, N, K
  GradientsPlan best;
  if (tokens == 0) return best;
  const Rate& rate = kRates[1];
  int64_t stages[3], longest = 0;
  double least = 0;  // of the products by themselves
  for (int i = 0; i < 3; ++i) {
    const int64_t M = sizes[i][0], N = sizes[i][1], K = sizes[i][2];
    stages[i] = (K + 63) / 64;
    longest = std::max(longest, stages[i]);
    least += product_time(i ? kTN : kNN, kStoreBf16, M, (int32_t)N, K, false);
  }
  for (int tile : {0, 3}) {
    const int64_t size = tile ? 64 : 128;
    int64_t tiles[3], all = 0;
    for (int i = 0; i < 3; ++i) {
      tiles[i] = ((sizes[i][0] + size - 1) / size) * ((sizes[i][1] + size - 1) / size);
      all += tiles[i];
    }
    if (all > 1024) continue;
    for (int64_t length = longest; length >= 2; length -= (length + 3) / 4) {
      GradientsPlan plan;
      plan.together = true;
      int64_t groups = 0;
      double work = 0, most = 0;
      for (int i = 0; i < 3; ++i) {
        Cut& c = plan.cut[i];
        const int64_t shares = (stages[i] + length - 1) / length;
        const int64_t share = (stages[i] + shares - 1) / shares;
        c = Cut{tile, (int)((stages[i] + share - 1) / share), (int)share, tiles[i]};
        c.time = share * rate.stage[tile] + rate.fixed[tile];
        groups += c.groups * c.shares;
        work += c.time * c.groups * c.shares / 256;
        most = std::max(most, c.time);
        plan.sums[i] = plan.bytes;
        if (c.shares > 1) plan.bytes += 4 * sizes[i][0] * sizes[i][1] * c.shares;
      }
      if (groups > 1024) break;
      const double time = (groups <= 256 ? most : work + most / 2) +
                          (plan.bytes ? 6.0 + 2 * plan.bytes / 4e6 : 0.0);
      if (time < least) least = time, best = plan;
    }
  }
  return best;
}

bool rows_fit(const Product& p, bool mx, AType a, bool paired) {
  const int64_t kb = mx ? p.K / 2 : 2 * p.K;
  return p.M >= 1 && p.M <= (a == kABf16 ? 16 : kMaxRows) &&
         (paired ? 2 : 1) * (int64_t)p.N * kb < 0x7fffffff &&
         (a == kAAsIs || p.M * ((int64_t)rows_code_stride(p.K) + rows_byte_stride(p.K)) <= kMxLds);
}

// Microseconds: a launch and a work-group's start and end, then what a CU spends
// on its work-groups' loads (a 16 x 64-byte load holds its address path 64
// cycles; MXFP4 with its scale bytes measured 240 a stage and tile), or the
// weights' way from memory; and the conversion of an fp32 A, about 280 cycles
// for each 16 bytes of a thread.
double rows_time(const Product& p, bool mx, AType a, bool paired) {
  const int64_t rows = (paired ? 2 : 1) * (int64_t)p.N, groups = (rows + 15) / 16;
  const int tiles = p.M <= 16 ? 1 : p.M <= 32 ? 2 : 4;
  const int64_t stages = (p.K + (mx ? 255 : 63)) / (mx ? 256 : 64);
  double cycles = (double)stages * (1 + tiles) * (mx ? 240 : 128);
  if (a == kAF32) cycles += (double)p.M * p.K / (4 * kRowsThreads) * 280;
  const double busy = (double)((groups + 255) / 256) * cycles / 2400;
  const double memory = (double)rows * p.K * (mx ? 0.53 : 2.0) / 4.5e6;
  return 4.0 + (busy > memory ? busy : memory);
}

}  // namespace ffn
