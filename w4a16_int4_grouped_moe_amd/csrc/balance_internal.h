// balance_internal.h -- what the balance loss's host code and kernels share.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

namespace balance {

constexpr int kMaxExperts = 1024;
constexpr int kWaves = 16;     // of a forward work-group
constexpr int kMostTokens = 64;  // tokens that a wave adds in fp32

struct Sizes {
  int64_t T;
  int32_t S, k, B, type;
};

// Tokens of a forward work-group: 16 waves of 1 to 64 tokens, 256 work-groups where
// there are as many; at most 128 tokens are one work-group's, which then ends the
// loss by itself.
constexpr int64_t kAlone = 128;
inline int64_t group_tokens(int64_t T) {
  if (T <= kAlone) return kAlone;
  const int64_t per = (T + 256 * kWaves - 1) / (256 * kWaves);
  return kWaves * std::min<int64_t>(per, kMostTokens);
}
inline int64_t groups(int64_t T) { return (T + group_tokens(T) - 1) / group_tokens(T); }
inline bool alone(const Sizes& z) { return z.B == 1 && z.T > 0 && z.T <= kAlone; }

// A work-group's part of a sequence is a piece: the sums of p (fp64 [S]), and the
// counts with the token count behind them (int32 [S + 1]). Piece of work-group g
// and sequence b: g + b, which no other pair has, since b never decreases with g.
inline int64_t pieces(const Sizes& z) { return groups(z.T) + z.B; }
inline int32_t column_groups(int32_t S) { return (S + 63) / 64; }
struct Workspace {
  size_t sums, counts, parts, bytes;  // parts: fp64 [B][column groups]
  explicit Workspace(const Sizes& z) {
    const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    sums = 0;
    counts = up((size_t)pieces(z) * z.S * 8);
    parts = counts + up((size_t)pieces(z) * (z.S + 1) * 4);
    bytes = alone(z) ? 0 : parts + up((size_t)z.B * column_groups(z.S) * 8);
  }
};

hipError_t launch_forward(const Sizes& z, const void* scores, const int32_t* ids,
                          const uint8_t* mask, const int32_t* offsets, float* loss,
                          int32_t* counts, int32_t* tokens, void* workspace, hipStream_t stream);
hipError_t launch_backward(const Sizes& z, const float* dloss, const void* scores,
                           const int32_t* counts, const int32_t* tokens, const uint8_t* mask,
                           const int32_t* offsets, void* dscores, hipStream_t stream);

}  // namespace balance
