// Which kernel form a layer operator's product runs, and its K splits: the
// rules behind gemm_layer.hip and gemm_layer_skinny.hip, with the measurements
// they rest on. Host only, no HIP: tests compile it by itself.
#pragma once

#include <stdint.h>

namespace fp8bl {
namespace plan {

constexpr int kTileK = 64;         // K of a 64-wide block (gemm_large_body.h)
constexpr int kTileCols = 256;     // weight rows of a tile, the gradient's output columns
constexpr int kStreamK = 256;      // K of a full super-step (gemm_skinny_body.h)
constexpr int kStreamWaves = 4;
constexpr int kStripCols = 256;    // output columns of the gradient's stream
constexpr int kStepRows = 32;      // and its weight rows a super-step

// Which of a product's two kernels runs: the streams of gemm_layer_skinny.hip
// (up to 32 rows) or the tiles. The streams start and end faster and keep more
// codes in flight; the tiles read X once a workgroup instead of once a wave.
// Measured on MI355X, stream against tiles, microseconds (graph replays that
// walk several weights, here and below):
//   linear  16 x 25600 x 5120  33.8  38.1    32 x 5120 x 5120   13.3  17.6
//           32 x 8000 x 8192   20.4  22.5    32 x 25600 x 5120  46.4  39.1
//   gated    8 x 25600 x 5120  49.9  63.1    16 x 25600 x 5120  56.0  66.9
//           16 x 5120 x 25600  71.6  60.2    32 x 8192 x 2048   14.3  16.9
//           32 x 5120 x 5120   23.8  20.6
//   input gradient (rows x weight rows x columns)
//           16 x 12288 x 4096  17.7  21.1    16 x 25600 x 5120  40.5  36
//           32 x 2048 x 4096   10.6  12.2    32 x 5120 x 5120   18.9  16.7
// (Pairs of nine to sixteen rows: past 2^27 codes the stream needs workgroups
// for two a CU, one per 16 columns.)
enum Product { kLinear, kPair, kInputGradient };
inline bool streams(Product p, int64_t m, int64_t n, int64_t codes) {
  if (m > 32) return false;
  switch (p) {
    case kLinear: return m <= 16 || codes <= (1 << 26);
    case kPair: return m <= 8 || codes <= (m <= 16 ? 1 << 27 : 1 << 25) || (m <= 16 && n >= 8192);
    default: return codes <= (m <= 16 ? 1 << 26 : 1 << 23);
  }
}

// ---- Tiles

// The tiles built: 32-row blocks of X, ring stages, 64-wide blocks of K per
// step; one workgroup a CU. (64 rows with 64 of K a step and two workgroups a
// CU: 64 x 25600 x 5120 47.4 us against 42.0, 64 x 5120 x 25600 45.3 against
// 38.2, 333 x 4304 x 1168 20.2 against 20.5.)
enum TileId { k256, k128, k64 };
template <int ID>
struct Tile;
template <>
struct Tile<k256> {
  static constexpr int kMB = 8, kStages = 3, kKS = 1;
};
template <>
struct Tile<k128> {
  static constexpr int kMB = 4, kStages = 4, kKS = 1;
};
template <>
struct Tile<k64> {
  static constexpr int kMB = 2, kStages = 3, kKS = 2;
};

// Tile and K splits of one of the three products: tiles of `cols` output
// columns, `products` sums over r, `words` fp32 partials an output (two for
// the gated pair). The model, in microseconds, was fitted to 3200 measurements
// of the three products on MI355X (48 to 512 rows, seven weights from 1024 x
// 1024 to 25600 x 5120, every tile, 1 to 24 splits; rms 6.5%, and the plan it
// picks is 2% slower than the best measured one on average, 16% at worst): a
// fixed part, then rounds of units over the chip, a step taking longer the
// more of the chip runs, then the join. (The pair was fitted with one array as
// both of its weights. With two, at 36 sizes of 40 to 512 rows, the plan is 1%
// slower than the best of three tiles and eight splits, 11% at worst.) Best of
// each tile, linear, us:
//    64 x 5120 x 5120   k64 19.2   k128 22.8   k256 25.2
//    64 x 5120 x 25600  k64 38.2   k128 45.3   k256 57.3
//   128 x 25600 x 5120  k64 56.7   k128 58.5   k256 72
//   512 x 25600 x 5120             k128 156    k256 122
struct LayerPlan {
  int tile;                                  // TileId
  int splits, steps_per_split;
  double cost;
};
struct TileCost {
  int tile, rows, k_step, stages;
  double fixed, step_few, step_full, unit;   // step_few: when few CUs run
};
template <int ID>
constexpr TileCost tile_cost(double fixed, double few, double full, double unit) {
  return TileCost{ID, 32 * Tile<ID>::kMB, kTileK * Tile<ID>::kKS, Tile<ID>::kStages, fixed, few, full, unit};
}
constexpr TileCost kTileCosts[] = {tile_cost<k256>(9.3, 1.07, 1.20, 0.5), tile_cost<k128>(8.9, 0.77, 0.84, 0.0),
                                   tile_cost<k64>(8.1, 1.03, 1.27, 0.0)};
constexpr int kCus = 256;
constexpr int kMaxSplits = 32;

// Steps of `products` sums over r, each padded to whole steps.
inline int64_t steps_of(int64_t r, int products, int k_step) { return (r + k_step - 1) / k_step * products; }

inline LayerPlan plan_tiles(int64_t m, int64_t n, int cols, int64_t r, int products, int words) {
  LayerPlan best{k256, 1, 0, 1e300};
  for (const TileCost& t : kTileCosts) {
    const int64_t tiles = ((m + t.rows - 1) / t.rows) * ((n + cols - 1) / cols);
    const int64_t steps = steps_of(r, products, t.k_step);
    for (int sp = 1; sp <= kMaxSplits; ++sp) {
      const int64_t per = (steps + sp - 1) / sp;
      if (sp > 1 && per * t.k_step < 4 * kTileK) break;
      const int64_t units = tiles * sp;
      const int64_t rest = units % kCus;
      double cost = t.fixed + (double)(units / kCus) * (per * t.step_full + t.unit);
      if (rest > 0) cost += per * (t.step_few + (t.step_full - t.step_few) * (double)rest / kCus) + t.unit;
      if (sp > 1) cost += 1.1 + 1e-6 * (double)(m * n) * (1.3 * sp * words + 1.0);
      if (cost < best.cost) best = LayerPlan{t.tile, (int)((steps + per - 1) / per), (int)per, cost};
    }
  }
  return best;
}

// A product as one or two launches over tile columns: where the tiles are a
// little more than whole rounds of the chip, the whole rounds run unsplit and
// only the columns left over are split (4096 x 12800 x 5120 backward, 320
// tiles: 256 unsplit and 64 in four instead of all 320 in four).
struct Part {
  int tile0, tiles_n;       // tile columns
  LayerPlan plan;
};
struct ProductPlan {
  int parts;
  Part part[2];
};
inline ProductPlan plan_product(int64_t m, int64_t n, int cols, int64_t r, int products, int words) {
  const int tn = (int)((n + cols - 1) / cols);
  ProductPlan best{1, {{0, tn, plan_tiles(m, n, cols, r, products, words)}, {}}};
  const TileCost& t = kTileCosts[k256];
  static_assert(kTileCosts[k256].tile == k256 && kTileCosts[k64].tile == k64, "the table is in the tiles' order");
  const int64_t steps = steps_of(r, products, t.k_step);
  const int64_t tm = (m + t.rows - 1) / t.rows;
  const int64_t rounds = tm * tn / kCus, head = rounds * kCus / tm;   // head: tile columns
  if (rounds > 0 && head < tn) {
    const LayerPlan h{t.tile, 1, (int)steps, t.fixed + (double)rounds * (steps * t.step_full + t.unit)};
    const LayerPlan rest = plan_tiles(m, n - head * cols, cols, r, products, words);
    if (h.cost + rest.cost < 0.98 * best.part[0].plan.cost)
      best = ProductPlan{2, {{0, (int)head, h}, {(int)head, (int)(tn - head), rest}}};
  }
  return best;
}

// ---- Streams

// How X is brought in (gemm_skinny_body.h), the K of a super-step, the ring's
// slots and the workgroups a CU holds. X goes through LDS, but for up to four
// rows of a gated pair or a small grid, where it is too little to matter.
// Half-width super-steps keep such a workgroup at 64 KB, two to a CU, where the
// grid has them, and leave 32 rows of X room for three slots. Microseconds, X
// in registers / through LDS in steps of 256 K / of 128 K, two to a CU:
//   linear   1 x 12288 x 4096  13.6    -   12.3    1 x 5120 x 25600  30.0    -   28.5
//           16 x 12288 x 4096  17.3  17.5  15.1   16 x 25600 x 5120  37.5  37.9  33.8
//           16 x 5120 x 5120   12.4  10.7  11.5   16 x 8000 x 8192   18.6  17.3  17.6
//            1 x 5120 x 5120    9.1   9.2    -     8 x 5120 x 5120   11.1  10.2  10.9
//   gated    1 x 25600 x 5120  46.9  54.5  48.2   16 x 12288 x 4096  25.8  26.8  22.5
//            8 x 25600 x 5120  49.5  59.7  50.1   16 x 2560 x 5120   12.1  10.7  11.4
// and of 17 to 32 rows, registers / LDS: linear 32 x 5120 x 5120 16.8 / 13.3,
// 32 x 4096 x 8192 22.2 / 17.1, gated 32 x 2560 x 5120 15.8 / 13.1,
// 32 x 8192 x 2048 16.8 / 14.3. (Four slots of 128 K: 12.3 at 16 x 5120 x 5120.)
template <int MT_, bool LDS_, int KW_, int D_, int RESIDENT_>
struct Path {
  static constexpr int MT = MT_, KW = KW_, D = D_, kResident = RESIDENT_;
  static constexpr bool kLds = LDS_;
};
template <typename F>
void with_path(int64_t m, int64_t workgroups, bool gated, F&& f) {
  if (m > 16) return f(Path<2, true, 128, 3, 1>{});
  const bool many = workgroups > 256;          // CUs get two
  if (m <= 4 && (gated || !many)) return f(Path<1, false, kStreamK, 2, 2>{});
  return many ? f(Path<1, true, 128, 2, 2>{}) : f(Path<1, true, kStreamK, 2, 1>{});
}

// Splits of the reduction: about two workgroups a CU (64 KB of LDS each), at
// least one super-step a wave.
struct GradientPlan {
  int strips, steps1, steps, splits, steps_per_split;
};
inline GradientPlan plan_gradient_skinny(int64_t n, int64_t k, int products) {
  GradientPlan p;
  p.strips = (int)((k + kStripCols - 1) / kStripCols);
  p.steps1 = (int)((n + kStepRows - 1) / kStepRows);
  p.steps = p.steps1 * products;
  int splits = (512 + p.strips - 1) / p.strips;
  const int most = (p.steps + kStreamWaves - 1) / kStreamWaves;
  if (splits > most) splits = most;
  p.steps_per_split = (p.steps + splits - 1) / splits;
  p.splits = (p.steps + p.steps_per_split - 1) / p.steps_per_split;
  return p;
}

// K splits of the two forward forms, by the workgroups (32 weight rows each)
// and a wave's super-steps. A split costs its join, about 3 us, so it has to
// save iterations: 16 x 5120 x 5120 (160 workgroups, 5 super-steps a wave)
// runs 12.2 us unsplit and 14.2 in two, 1 x 2048 x 2048 5.0 and 5.9; but
// 1 x 1024 x 8192 (32 workgroups, 8 super-steps) 10.8 unsplit and 7.1 in four,
// and 16 x 5120 x 25600 (25 super-steps, 160 workgroups on 256 CUs) 42.7
// unsplit and 37.9 in four.
struct StreamPlan {
  int splits, ss_per_split;
};
inline StreamPlan plan_layer(int64_t groups, int64_t k) {
  const int nss = (int)((k + kStreamK - 1) / kStreamK);
  const int iters = (nss + kStreamWaves - 1) / kStreamWaves;
  int splits = 1;
  if (groups < 128 && iters >= 4) {
    while (groups * splits < 128 && splits * 2 <= iters) splits *= 2;
  } else if (groups < 256 && iters >= 16) {
    splits = 4;
  }
  StreamPlan p;
  p.ss_per_split = (nss + splits - 1) / splits;
  p.splits = (nss + p.ss_per_split - 1) / p.ss_per_split;
  return p;
}

}  // namespace plan
}  // namespace fp8bl
