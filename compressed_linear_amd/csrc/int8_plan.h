// int8_plan.h -- how the product in 8-bit integers is cut into tiles and parts of K, by its sizes alone (host code).
#pragma once
#include <stdint.h>

#include <algorithm>

namespace cl {
namespace {

inline int64_t padded(int64_t K) { return (K + 127) / 128 * 128; }

constexpr int kCus = 256;
constexpr int kMostParts = 16;

// What int8_stream_kernel takes: up to 16 tokens, and up to 64 with few weights, where reading the tokens once for every 16 outputs costs
// less than the start of tiles (32 tokens of 4096 x 4096 6.9 us, as tiles 10.1; 64 tokens 8.8 and 11.3; past that 32 tokens of
// 4096 x 11008 14.6 and 13.0, 64 of them 20.2 and 14.6, 64 of 11008 x 4096 17.9 and 16.2).
inline bool streamed(int tokens, int N, int K) { return tokens <= 16 || (tokens <= 64 && (int64_t)N * K <= 1 << 25); }

// How a product is cut: the tile, parts of K.
struct Plan {
  int shape = 0, parts = 1;
};

// Tiles, and what they cost: the microseconds that a step of 128 k takes a CU for each tile that it has, and how many of them run at
// once.  The costs were fitted to the times of whole products, so that waits for weights that no other tile reads are in them; in a long run of
// rows that 16 tiles share a step takes 1.60, 1.32, 0.90 (1.14 with two buffers), 0.60, 0.48, 0.31 and 0.25 us.  Small tiles run side by side
// and fill in for each other, but read more for what they multiply.
struct Shape {
  int tw, tt, together;
  float step;
};
constexpr Shape kShapes[] = {{256, 256, 1, 1.72f}, {256, 192, 1, 1.45f}, {256, 128, 1, 1.19f}, {128, 128, 1, 0.54f},
                             {128, 64, 2, 0.46f},  {64, 64, 2, 0.265f},  {64, 32, 3, 0.235f}};
constexpr int kShapeCount = sizeof kShapes / sizeof kShapes[0], kHalf = 2;

inline int64_t tiles_of(const Shape& s, int tokens, int N) { return (((int64_t)tokens + s.tt - 1) / s.tt) * ((N + s.tw - 1) / s.tw); }

// Half of the last round's tiles or fewer: each is cut in two, with a buffer more, so that the round is shorter (2048 x 8192 x 28672 has 3.5
// rounds: 415 us, with whole tiles 440).
inline bool halved(int64_t tiles) { return tiles % kCus && tiles % kCus <= kCus / 2; }

// The cheapest of the tiles and parts of K by those costs: steps x tiles of the busiest CU, 3.5 us to fill and to empty each, at least the
// time to read the weights (8 TB/s is more than memory gives: it ranks the small products), and for parts 4 us and the sums
// written and read at 4.2 TB/s.  Over 97 products of 24 to 4096 tokens and 1000 x 1000 to 8192 x 28672 weights the choice
// is 2 % slower than the best of all in the mean and 29 % at worst (where 256 x 128 tiles would do better than their cost says); 256 x 256 tiles
// without parts take up to 4.3 times as long as the best.
inline Plan plan_product(int tokens, int N, int K) {
  Plan best;
  if (tiles_of(kShapes[0], tokens, N) > 4 * kCus) return best;
  const int steps = (int)(padded(K) / 128);
  float least = 1e30f;
  for (int shape = 0; shape < kShapeCount; ++shape) {
    const Shape& s = kShapes[shape];
    const int64_t tiles = tiles_of(s, tokens, N);
    for (int parts = 1; parts <= kMostParts && parts <= (steps + 3) / 4; ++parts) {
      const int64_t n = tiles * parts;
      if (parts > 1 && n > 4 * kCus) break;
      const int each = (steps + parts - 1) / parts;
      const bool half = shape == 0 && halved(n);
      const int64_t whole = half ? n / kCus : (n + kCus - 1) / kCus;
      float t = each * (whole * s.step + (half ? kShapes[kHalf].step : 0)) + 3.5f * ((whole + s.together - 1) / s.together + half);
      t = std::max(t, (float)N * K / 8e6f);
      if (parts > 1) t += 4.f + 4.f * tokens * N * parts / 4.2e6f;
      if (t < least) least = t, best = Plan{shape, parts};
    }
  }
  return best;
}

}  // namespace
}  // namespace cl
