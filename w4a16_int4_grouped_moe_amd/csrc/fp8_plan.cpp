// fp8_plan.cpp -- which tiles compute an FP8 product: host arithmetic on the sizes,
// by times measured on the MI355X.
#include "fp8_internal.h"

namespace fp8 {
namespace {

// Microseconds a stage of K takes one round of work-groups on 256 CUs, and what a
// work-group costs besides, its launch among it; by tile (see Cut). Measured on one
// round of each tile at K of 1024 and 4096: [wide][B in 1 x 128 blocks].
struct Rate {
  double stage[4], fixed[4];
};
constexpr Rate kRates[2][2] = {{{{0.78, 0.89, 1.53, 0.32}, {6.4, 8.6, 13.9, 5.3}},
                                {{0.91, 1.19, 2.28, 0.31}, {5.7, 7.5, 12.5, 5.4}}},
                               {{{1.20, 1.66, 9.00, 0.49}, {7.4, 10.7, 20.0, 4.6}},
                                {{1.27, 1.84, 9.00, 0.49}, {8.2, 10.2, 20.0, 4.4}}}};

}  // namespace

// The cheapest cut. Shares of K cost a launch and the sums' way to memory and
// back (about 4 TB/s); of equals the larger tile.
Cut cut_of(bool wide, bool rows, int64_t M, int64_t N, int64_t K) {
  const Rate& rate = kRates[wide][rows];
  const int64_t stages = blocks_of(K);
  const auto tiles = [&](int64_t high, int64_t across) {
    return ((M + high - 1) / high) * ((N + across - 1) / across);
  };
  const auto time = [&](int tile, int64_t groups, int64_t st) {
    return (double)((groups + 255) / 256) * (st * rate.stage[tile] + rate.fixed[tile]);
  };
  const int64_t n[4] = {tiles(128, 128), tiles(128, 256), tiles(256, 256), tiles(64, 64)};
  Cut best{1, 1, (int)stages, n[1], time(1, n[1], stages)};
  if (const double t = time(2, n[2], stages); !wide && t <= best.time)
    best = Cut{2, 1, (int)stages, n[2], t};
  for (int tile : {0, 3})
    for (int shares = 1; shares <= 32 && n[tile] * shares <= 1024; ++shares) {
      const int64_t share = (stages + shares - 1) / shares;
      if (shares > 1 && (2 * shares > stages || share * (shares - 1) >= stages)) continue;
      const double t = time(tile, n[tile] * shares, share) +
                       (shares > 1 ? 3.0 + 8.0 * M * N * shares / 4e6 : 0);
      if (t < best.time) best = Cut{tile, shares, (int)share, n[tile], t};
    }
  return best;
}

// A product whose last round of the largest tiles is nearly empty takes two launches: its first
// rows in whole rounds, the rest cut on its own. Measured, whole calls on codes, one launch and
// two: 4352 x 4096 x 4096 93 -> 75 us (fp32 results 169 -> 139), 5120 x 4096 x 7168 157 -> 146
// (293 -> 267), 2304 x 8192 x 1024 37.8 -> 34.3 (59 -> 57). The second launch counts 3 us, and an
// estimate less than 5% lower is within the estimates' error and stays one launch. With B in 1 x 128
// blocks and bf16 results a nearly empty round takes less than it is counted for: two launches that
// were estimated 13% lower took 62 -> 66 us (2560 x 7168 x 2048), 23% lower 79 -> 63 (2307 x 6840 x
// 2544).
Plan plan_of(bool wide, bool rows, int64_t M, int64_t N, int64_t K) {
  Plan best;
  best.whole = cut_of(wide, rows, M, N, K);
  best.time = best.whole.time;
  const int tile = wide ? 1 : 2;
  const int64_t high = wide ? 128 : 256, tn = (N + 255) / 256;
  const int64_t rounds = ((M + high - 1) / high * tn + 255) / 256;
  if (rounds < 2) return best;
  const int64_t first = (rounds - 1) * 256 / tn * high;  // of whole rounds
  if (first <= 0 || first >= M) return best;
  const Rate& rate = kRates[wide][rows];
  const int64_t stages = blocks_of(K), groups = first / high * tn;
  const Cut whole{tile, 1, (int)stages, groups,
                  (double)((groups + 255) / 256) * (stages * rate.stage[tile] + rate.fixed[tile])};
  const Cut rest = cut_of(wide, rows, M - first, N, K);
  const double both = whole.time + rest.time + 3.0;
  if (both < (rows && !wide ? 0.85 : 0.95) * best.time)
    best.first = first, best.whole = whole, best.rest = rest, best.time = both;
  return best;
}

// Microseconds of the few-row kernel: rounds of work-groups on 256 CUs, each a work-group's start
// and end and its stages. Measured, and beside it 64 x 64 tiles with shares of K, in whole calls on
// codes: 4096 x 7168 with 1, 8 and 16 rows 8.9, 9.8, 11.8 (tiles 12 to 12.7), 4096 x 28672 22.3, 24.5,
// 29.4 (27.5), 7168 x 2048 9.2, 11.1, 13.8 (9.1 to 9.4); with 32 rows, which the kernel does not
// take, it was 15.0 where tiles were 13.0.
double rows_time(int64_t M, int64_t N, int64_t K) {
  const int64_t groups = (N + 15) / 16;
  return (double)((groups + 255) / 256) * (4.5 + (0.075 + 0.0035 * M) * blocks_of(K));
}

size_t product_workspace(bool wide, bool rows, int64_t M, int32_t N, int64_t K) {
  if (M == 0) return 0;
  const Plan plan = plan_of(wide, rows, M, N, K);
  const Cut& c = plan.first ? plan.rest : plan.whole;
  return c.shares > 1 ? (size_t)c.shares * (M - plan.first) * N * 4 : 0;
}

}  // namespace fp8
