// Prints how products are cut: for each line "ffn T H I", "mxffn T H I" or "mx M
// N K" on stdin one line of "name first rest-or-whole": name, the rows of a first
// launch (0: one launch), the tile of the rest (or the whole) and its shares of K.
#include <cstdio>
#include <cstring>

#include "ffn_internal.h"

namespace {
void print(const char* name, ffn::Layout l, ffn::Epilogue e, int64_t M, int64_t N, int64_t K, bool mx) {
  const ffn::Plan p = ffn::plan_of(e, M, N, K, l, mx);
  const ffn::Cut& c = p.first ? p.rest : p.whole;
  std::printf("%s %lld %d %d; ", name, (long long)p.first, c.tile, c.shares);
}
}  // namespace

int main() {
  char kind[16];
  long long a, b, c;
  while (std::scanf("%15s %lld %lld %lld", kind, &a, &b, &c) == 4) {
    if (!std::strcmp(kind, "mx")) {
      print("product", ffn::kNT, ffn::kStoreF32, a, b, c, true);
    } else {
      const bool mx = !std::strcmp(kind, "mxffn");
      print("up", ffn::kNT, mx ? ffn::kSwigluMx : ffn::kSwiglu, a, c, b, mx);
      print("down", ffn::kNT, ffn::kStoreBf16, a, b, c, mx);
      if (!mx) {
        print("dh", ffn::kNN, ffn::kSwigluGrad, a, c, b, false);
        if (!ffn::gradients_plan(a, b, c).together) {
          print("dx", ffn::kNN, ffn::kStoreBf16, a, b, 2 * c, false);
          print("dw13", ffn::kTN, ffn::kStoreBf16, 2 * c, b, a, false);
          print("dw2", ffn::kTN, ffn::kStoreBf16, b, c, a, false);
        }
      }
    }
    std::printf("\n");
  }
}
