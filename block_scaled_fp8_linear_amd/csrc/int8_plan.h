// How the 8-bit integer linear is cut: tiles and K splits of gemm_int8.hip, the
// workgroups of gemm_int8_skinny.hip, with the measurements the rules rest on.
// Host only, no HIP: tests compile it by itself.
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace fp8bl {

constexpr int64_t kInt8SkinnyRows = 32;      // most rows of gemm_int8_skinny.hip
constexpr int kInt8FusedK = 16384;           // of one row that the product's own workgroups quantize

// One row of up to 16384, which the threads' registers hold.
inline bool int8_skinny_quantizes(int64_t m, int64_t k) { return m == 1 && k <= kInt8FusedK; }

// How a workgroup is cut, by the row tiles of X (m > 16) and whether 16 weight
// rows a workgroup still leave no compute unit a second one (few).
//
// With few columns (n <= 4096): 16 rows by eight waves (four for two row tiles of
// X): 1 x 4000 x 8192 takes 7.4 us so, 9.9 in 32 rows by four waves; 1 x 1000 x
// 8192 5.8 and 8.1. Otherwise several workgroups share a compute unit, for which
// super-steps of 128 or few waves leave the LDS: 16 x 25600 x 5120 takes 26.5 us
// in 32 rows, four waves and super-steps of 128, 33.0 with super-steps of 256 (one
// workgroup a compute unit, 800 of them), 31.7 in 16 rows by eight waves; one row
// in 16 rows by four waves 25600 x 5120 25.8, 8000 x 8192 12.0 (14.5 in 32 rows).
//
// K is split over workgroups from 16384 on (8192 with two row tiles), in pieces
// of 2048 or more, as far as there are compute units for them: the join costs
// 2.5 us, 16 x 300 x 25600 takes 17.5 us whole and 7.7 in eight, 16 x 2000 x 8192
// 8.0 and 8.2 in two. Not for a row of bf16 that is quantized on the way: its
// quantizer would need a launch of its own.
struct Int8SkinnyPlan {
  bool few;
  int splits, k_split;
};
inline Int8SkinnyPlan plan_skinny8(int64_t m, int64_t n, int64_t k) {
  const int64_t groups = (n + 15) / 16;
  Int8SkinnyPlan p{groups <= 256, 1, 0};
  if (k >= (m > 16 ? 8192 : 16384) && !int8_skinny_quantizes(m, k))
    while (groups * p.splits * 2 <= 256 && k >= 4096 * (int64_t)p.splits) p.splits *= 2;
  p.k_split = (int)((k + 256 * p.splits - 1) / (256 * p.splits)) * 256;      // whole super-steps of either size
  p.splits = (int)((k + p.k_split - 1) / p.k_split);
  return p;
}

constexpr int kInt8Edge[3] = {256, 128, 64};
constexpr int kInt8StepK = 128;              // K of a step of the tiles

struct Int8Plan {
  int tile;        // of kInt8Edge
  int splits;
};

// Tile edge and split count by a time estimate in microseconds, fitted to 21
// shapes from 48 x 8000 x 8192 to 2000 x 256 x 25600 measured with every choice: a
// step of 128 of K on a compute unit, a unit's start and epilogue, and the join of
// splits (large tiles have become a little faster since; on 13 shapes measured again
// the choices are at most 3% above the best). Units of 64 run two to a compute unit.
// 512 x 5120 x 5120 takes 24.9 us in tiles of 128, 31.3 of 64 and 55.8 of 256;
// 333 x 4300 x 1168 11.4, 9.0 and 25.6; 2048 x 5120 x 5120 66.9, 90.8 and 57.5;
// 4096 x 4096 x 4096 77.2, 114 and 60.2; 64 x 1000 x 25600 57.6 in tiles of 64 and
// 13.4 with eight splits.
inline Int8Plan plan_int8(int64_t m, int64_t n, int64_t k) {
  constexpr double kStepUs[3] = {1.8, 0.61, 0.33}, kUnitUs[3] = {5.0, 2.2, 1.1};
  constexpr double kJoinUs = 2.2, kJoinElemUs = 2.1e-6;
  const int64_t steps = (k + kInt8StepK - 1) / kInt8StepK;
  Int8Plan best{0, 1};
  double least = 1e300;
  for (int t = 0; t < 3; ++t) {
    const int64_t tiles = ((m + kInt8Edge[t] - 1) / kInt8Edge[t]) * ((n + kInt8Edge[t] - 1) / kInt8Edge[t]);
    for (const int splits : {1, 2, 3, 4, 6, 8}) {
      const int64_t each = (steps + splits - 1) / splits;
      if (splits > 1 && each < 4) break;
      const int64_t units = tiles * splits;
      double us;
      if (t == 2) {
        const int64_t rest = units % 512;
        us = (double)(2 * (units / 512) + (rest == 0 ? 0 : rest <= 256 ? 1 : 2)) * each * kStepUs[t] +
             (double)((units + 511) / 512) * kUnitUs[t];
      } else {
        us = (double)((units + 255) / 256) * (each * kStepUs[t] + kUnitUs[t]);
      }
      if (splits > 1) us += kJoinUs + kJoinElemUs * splits * (double)m * (double)n;
      if (us < least) {
        least = us;
        best = Int8Plan{t, splits};
      }
    }
  }
  return best;
}

// A product cut by its plan: tiles, and steps of K to each split, of which none is
// empty. In 64 bits: m reaches 2^31 - 1.
struct Int8Cut {
  int64_t tiles_m, tiles_n, steps, steps_per_unit, splits, units;
};
inline Int8Cut cut_int8(int64_t m, int64_t n, int64_t k, int edge, int splits) {
  Int8Cut c;
  c.tiles_m = (m + edge - 1) / edge;
  c.tiles_n = (n + edge - 1) / edge;
  c.steps = (k + kInt8StepK - 1) / kInt8StepK;
  c.steps_per_unit = (c.steps + splits - 1) / splits;
  c.splits = (c.steps + c.steps_per_unit - 1) / c.steps_per_unit;
  c.units = c.tiles_m * c.tiles_n * c.splits;
  return c;
}

}  // namespace fp8bl
