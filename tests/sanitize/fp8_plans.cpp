// Prints how FP8 products are cut: for each line "wide rows M N K" on stdin one line
// of the rows of a first launch (0: there is one launch) and the tile and shares of K of the
// rest.
#include <cstdio>

#include "fp8_internal.h"

int main() {
  long long wide, rows, M, N, K;
  while (std::scanf("%lld %lld %lld %lld %lld", &wide, &rows, &M, &N, &K) == 5) {
    const fp8::Plan p = fp8::plan_of(wide != 0, rows != 0, M, N, K);
    const fp8::Cut& c = p.first ? p.rest : p.whole;
    std::printf("%lld %d %d\n", (long long)p.first, c.tile, c.shares);
  }
}
