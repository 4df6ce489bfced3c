// The choice of a product's tile and split (kernels_linear.hip launches what it says). Host code
// without HIP, so that the choice can be asked for without a device.
#pragma once

#include <algorithm>

namespace instant {

// Tile (wm, wn: 16-row tiles of a wave; a block is 32 wm x 32 wn), stages held in LDS and K
// slices of a product.
struct Plan {
  int wm, wn, ns, S;
  bool part;  // float32 partials instead of the output (S > 1 needs it)
  bool add;   // added to those that are there
};

namespace planning {

// A product's time by what its blocks cost: a compute unit runs `fit` blocks of a shape at once;
// a block takes at least `lone` us a stage (the latency of its requests), k of them together at
// least k * `each` (the matrix cores and the operands' way to them), and `ends` for its start and
// its epilogue. Split K pays for a second launch and the partials' way to memory and back.
//
// The figures are fitted to measured times on gfx950 of 69 products in bfloat16 (three layouts, 1
// to 16384 rows, columns and k) and 51 in float32, by 9 tile shapes and ring depths by 8 splits.
// The choice is within 5% of the best of all measured in 66 of the 69 (1.4% behind on average)
// and in 42 of the 50 whose choice was measured (3.4%; 20 x 3000 over 1000 is 15.7 against 10.3 us).
// What the choice is worth in bfloat16, best against a fixed 256 x 256
// tile: 8 x 11008 over 4096 15.0 against 73 us, 768 x 768 over 16384 40 against 309 us, 512 x 4096
// over 1024 8.5 against 31 us; against a fixed 64 x 64 tile: 16384 x 1024 over 4096 108 against
// 197 us. In float32 the matrix cores have an eighth of the rate, nothing else holds them up, and
// four shapes do.
//
// An epilogue with an activation or a checkpoint (`heavy`: up to 60 operations a value) costs
// tiles that have a compute unit to themselves more: nothing runs beside it. (bfloat16 with
// GELU and an 8-bit pre-activation, 256 x 192 against 128 x 128 tiles: 16384 x 768 over 768 35.5
// against 33.0 us, without them 26.3 against 27.7; 6272 x 1792 over 448 29.9 against 25.3 us; but
// 16384 x 11008 over 4096, whose stages outweigh it, 1212 with 256 x 256 against 1515 us.) The two
// factors are shared by all shapes, and the 128 x 128 tile with two blocks a unit costs more over
// long contractions than the rule says: M x 11008 over 4096 with GELU and an 8-bit pre-activation
// takes 128 x 128 for M = 4096, 8192, 12288 and 14336 (349, 769, 1138 and 1232 us) where 256 x 256
// is faster (331, 651, 964 and 1087).
struct Shape {
  int wm, wn, ns, fit;
  float lone, each, ends;
};
constexpr Shape SHAPES_BF16[] = {
    {8, 8, 2, 1, 1.21f, 1.17f, 8.4f},  {8, 6, 2, 1, 1.01f, 0.91f, 7.4f},   {4, 4, 2, 2, 0.47f, 0.356f, 2.14f},
    {4, 4, 4, 1, 0.43f, 0.25f, 3.0f},  {2, 4, 3, 2, 0.33f, 0.253f, 2.67f}, {2, 2, 2, 4, 0.43f, 0.204f, 0.84f},
    {2, 2, 4, 2, 0.05f, 0.192f, 1.91f}, {1, 2, 4, 3, 0.07f, 0.176f, 1.13f}};
constexpr Shape SHAPES_FP32[] = {{8, 8, 2, 1, 1.0f, 7.5f, 7.9f},
                                 {4, 4, 2, 2, 2.16f, 1.9f, 2.8f},
                                 {2, 2, 2, 4, 0.62f, 0.505f, 1.26f},
                                 {1, 2, 4, 3, 0.37f, 0.29f, 1.1f}};

template <int NSH> inline Plan choose(const Shape (&shapes)[NSH], int nst, int M, int N, bool heavy) {
  static constexpr int slices[] = {1, 2, 3, 4, 6, 8, 12, 16};
  Plan best{0, 0, 0, 1, false, false};
  float least = 0.0f;
  for (const Shape& s : shapes) {
    const float ends = s.ends * (!heavy ? 1.0f : s.fit == 1 ? 2.6f : 2.0f);
    const long tiles = (((long)M + 32 * s.wm - 1) / (32 * s.wm)) * (((long)N + 32 * s.wn - 1) / (32 * s.wn));
    for (int S : slices) {
      if (S > 1 && (tiles * S > 2048 || nst < 2 * S)) break;
      const long n = (tiles * S + 255) / 256;  // blocks of the busiest compute unit
      const int nq = (nst + S - 1) / S;
      auto group = [&](int k) { return nq * std::max(s.lone, k * s.each) + ends * (0.5f + 0.5f * k); };
      const int rest = (int)(n % s.fit);
      float t = (float)(n / s.fit) * group(s.fit) + (rest ? group(rest) : 0.0f);
      if (S > 1) t += 2.0f + 0.1f * S + (float)S * M * N * 8.0f / 7.6e6f;
      if (!best.wm || t < least) {
        best = Plan{s.wm, s.wn, s.ns, S, S > 1, false};
        least = t;
      }
    }
  }
  return best;
}

}  // namespace planning

// An M x N output over K; heavy: with an activation or a checkpoint in its epilogue.
inline Plan plan(bool bf16_io, int M, int N, int K, bool heavy) {
  using namespace planning;
  return bf16_io ? choose(SHAPES_BF16, (K + 63) / 64, M, N, heavy) : choose(SHAPES_FP32, (K + 31) / 32, M, N, heavy);
}

}  // namespace instant
