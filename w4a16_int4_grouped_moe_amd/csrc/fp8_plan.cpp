// fp8_plan.cpp -- which tiles compute an FP8 product: host arithmetic on the sizes,
// by times measured on the MI355X.
#include "fp8_internal.h"

namespace fp8 {
namespace {

// Microseconds a stage of K takes one round of work-groups on 256 CUs, and what a
// work-group costs besides; by tile (see Cut), narrow and wide.
struct Rate {
  double stage[4], fixed[4];
};
constexpr Rate kRates[2] = {{{0.62, 0.88, 1.42, 0.32}, {4.5, 4.5, 7.0, 4.5}},
                            {{0.90, 1.60, 9.00, 0.40}, {4.5, 5.0, 7.0, 4.5}}};

}  // namespace

// The cheapest cut. Shares of K cost a launch and the sums' way to memory and
// back (about 4 TB/s); of equals the larger tile.
Cut cut_of(bool wide, int64_t M, int64_t N, int64_t K) {
  const Rate& rate = kRates[wide];
  const int64_t stages = blocks_of(K);
  const auto tiles = [&](int64_t rows, int64_t cols) {
    return ((M + rows - 1) / rows) * ((N + cols - 1) / cols);
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

// Microseconds: a launch and a work-group's start and end, then what a CU spends on its
// work-groups' loads (a 16 x 64-byte load of A holds its address path 64 cycles, a line of B
// 18 for 8 rows), or the weights' way from memory.
double rows_time(int64_t M, int64_t N, int64_t K) {
  const int64_t groups = (N + 15) / 16;
  const int tiles = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  const double busy = (double)((groups + 255) / 256) * blocks_of(K) * (36 + 128 * tiles) / 2400;
  const double memory = (double)N * K / 4.5e6;
  return 5.0 + (busy > memory ? busy : memory);
}

size_t product_workspace(bool wide, int64_t M, int32_t N, int64_t K) {
  if (M == 0) return 0;
  const Cut c = cut_of(wide, M, N, K);
  return c.shares > 1 ? (size_t)c.shares * M * N * 4 : 0;
}

}  // namespace fp8
