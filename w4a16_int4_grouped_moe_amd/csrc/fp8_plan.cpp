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
  const Cut c = cut_of(wide, rows, M, N, K);
  return c.shares > 1 ? (size_t)c.shares * M * N * 4 : 0;
}

}  // namespace fp8
