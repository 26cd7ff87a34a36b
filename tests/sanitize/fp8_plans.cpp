// Prints how FP8 products are cut: for each line "wide rows M N K" on stdin one line
// of the tile and its shares of K.
#include <cstdio>

#include "fp8_internal.h"

int main() {
  long long wide, rows, M, N, K;
  while (std::scanf("%lld %lld %lld %lld %lld", &wide, &rows, &M, &N, &K) == 5) {
    const fp8::Cut c = fp8::cut_of(wide != 0, rows != 0, M, N, K);
    std::printf("%d %d\n", c.tile, c.shares);
  }
}
