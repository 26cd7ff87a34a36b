// fp8_rows_plan.cpp -- which sizes the few-row FP8 kernels take, and what a work-group
// of theirs takes: host arithmetic on the sizes.
#include "fp8_internal.h"

namespace fp8 {
namespace {
constexpr int64_t kMostExtra = 64 * 1024;  // LDS beside the ring
}

int64_t rows_extra(bool fresh, int64_t rows, int64_t K, int slices) {
  return rows_sums_at(fresh, rows, K) + (fresh ? slices * kRowsWaves * rows * 64 : 0);
}

bool rows_fit(Source source, int64_t M, int64_t N, int64_t K) {
  return M >= 1 && M <= (source == kCodes ? kMostRows : kFewRows) && N < (1 << 26) &&
         N * K <= 0x7fffffff && rows_extra(source != kCodes, M, K, 1) <= kMostExtra;
}

// As many slices as leave two work-groups for every CU, and two on it (N is a multiple of 128, and
// a work-group's columns lie in one block)
int experts_slices(Epilogue epilogue, int64_t N, int64_t K, int64_t buckets) {
  const int64_t all = (N + rows_step(epilogue) - 1) / rows_step(epilogue);
  int slices = 1;
  while (slices < 8 && all / (2 * slices) * buckets >= 512 &&
         rows_extra(true, kFewRows, K, 2 * slices) + kExpertsStages * kRowsWaves * kRowsSlot <=
             80 * 1024)
    slices *= 2;
  return slices;
}

}  // namespace fp8
