// Kernels of the layer operators (fp8bl_layers.h) above the rows that stream
// (gemm_layer_skinny.hip): the epilogues on the large-M kernel's loop
// (gemm_large_body.h) and the input gradient, whose reduction runs over the
// weight's rows.
//
// All three are products of m rows with the decoded weight, sums in fp32. With
// many rows the matrix instructions bound them, at 1.2 to 1.3 PFLOP/s, where
// the plain linear on the same loop reaches 1.29 and a bf16 library product of
// 8192^3 1.46: the MFMAs are busy 64 to 73% of the cycles (the issue of the
// loads takes the rest) and the clock falls to 1.5 - 1.7 GHz. At some hundred
// rows it is what a launch cannot spread: a tile costs about 9 us before its
// first and after its last step, and tiles rarely fill whole rounds of 256 CUs.
// At tens of rows it is the codes' bytes.
#include "gemm_large_body.h"

namespace fp8bl {

namespace {

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

struct Grid {
  int gk, tiles_m, tiles_n, steps, splits, steps_per_unit;
};

// y = act(x W^T + bias) + residual, and z = x W^T + bias where it is saved:
// bias, activation and residual on the fp32 sums in the epilogue, so that z is
// written once and nothing is read back. (8192 x 12288 x 4096 with bias, tanh
// GELU and z saved 672 - 695 us, 1.19 - 1.23 PFLOP/s; y alone, plain, 630.
// 512 x 5120 x 25600 with residual 129 us, 1.04 PFLOP/s; 512 x 5120 x 5120 41
// us, of which the join of its splits is 7.)
template <bool SPLIT, int ACT, int ID>
__global__ __launch_bounds__(kThreads, 1)
void linear_act_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ q,
                       const float* __restrict__ s, uint16_t* y, float* __restrict__ part, int M, int N,
                       int K, Grid g, LargeArgs la) {
  gemm_large_body<SPLIT, false, kLayer, ACT, Tile<ID>::kMB, Tile<ID>::kStages, Tile<ID>::kKS>(
      x, q, s, nullptr, nullptr, y, part, M, N, K, g.gk, g.tiles_m, g.tiles_n, g.steps, g.splits,
      g.steps_per_unit, la);
}

// h = act(x Wg^T) (x Wu^T): a tile is 128 output columns, and each wave holds
// gate and up of the same 32 of them, so that the product needs no exchange
// between waves and both sums are whole in fp32 when it is taken. (512 x 25600
// x 5120 with g and u saved 248 us, 1.08 PFLOP/s: 400 tiles on 256 CUs are 78%
// of two rounds.)
template <bool SPLIT, int ACT, int ID>
__global__ __launch_bounds__(kThreads, 1)
void glu_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ qg, const float* __restrict__ sg,
                const uint8_t* __restrict__ qu, const float* __restrict__ su, uint16_t* __restrict__ h,
                float* __restrict__ part, int M, int N, int K, Grid g, LargeArgs la) {
  gemm_large_body<SPLIT, false, kGlu, ACT, Tile<ID>::kMB, Tile<ID>::kStages, Tile<ID>::kKS>(
      x, qg, sg, qu, su, h, part, M, N, K, g.gk, g.tiles_m, g.tiles_n, g.steps, g.splits, g.steps_per_unit, la);
}

// dx = x W (+ x2 W2): C output columns, R weight rows. The weight's rows are
// the reduction: codes come in as [row][column] and transposing LDS reads
// (ds_read_b64_tr_b8) hand each lane eight rows of its column, so neither a
// transposed copy of the weight nor a shuffle is needed, and one decode per
// code feeds the tile's rows as in the forward. The two products of the gated
// backward are one reduction of twice the length: one launch, one rounding.
// (dx of 4096 x 12288 x 4096 311 - 323 us, 1.28 PFLOP/s and more; of the pair 4096 x 12800 x
// 5120 851 us with the join, 1.26 PFLOP/s.)
template <bool SPLIT, int ID>
__global__ __launch_bounds__(kThreads, 1)
void input_gradient_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ q,
                           const float* __restrict__ s, const uint8_t* __restrict__ q2,
                           const float* __restrict__ s2, uint16_t* __restrict__ dx,
                           float* __restrict__ part, int M, int C, int R, Grid g, LargeArgs la) {
  gemm_large_body<SPLIT, false, kGradient, kActNone, Tile<ID>::kMB, Tile<ID>::kStages, Tile<ID>::kKS>(
      x, q, s, q2, s2, dx, part, M, C, R, g.gk, g.tiles_m, g.tiles_n, g.steps, g.splits, g.steps_per_unit, la);
}

int blocks_of(int64_t v) { return (int)((v + kBlock - 1) / kBlock); }

// Tile and K splits of one of the three products: tiles of `cols` output
// columns, `products` sums over r, `words` fp32 partials an output (two for
// the gated pair). The model, in microseconds, was fitted to 3200 measurements
// of the three products on MI355X (48 to 512 rows, seven weights from 1024 x
// 1024 to 25600 x 5120, every tile, 1 to 24 splits; rms 6.5%, and the plan it
// picks is 2% slower than the best measured one on average, 16% at worst): a
// fixed part, then rounds of units over the chip, a step taking longer the
// more of the chip runs, then the join. Best of each tile, linear, us:
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
  return TileCost{ID, 32 * Tile<ID>::kMB, kBK * Tile<ID>::kKS, Tile<ID>::kStages, fixed, few, full, unit};
}
constexpr TileCost kTileCosts[] = {tile_cost<k256>(9.3, 1.07, 1.20, 0.5), tile_cost<k128>(8.9, 0.77, 0.84, 0.0),
                                   tile_cost<k64>(8.1, 1.03, 1.27, 0.0)};
constexpr int kCus = 256;
constexpr int kMaxSplits = 32;

// Steps of `products` sums over r, each padded to whole steps.
int64_t steps_of(int64_t r, int products, int k_step) { return (r + k_step - 1) / k_step * products; }

LayerPlan plan_tiles(int64_t m, int64_t n, int cols, int64_t r, int products, int words) {
  LayerPlan best{k256, 1, 0, 1e300};
  for (const TileCost& t : kTileCosts) {
    const int64_t tiles = ((m + t.rows - 1) / t.rows) * ((n + cols - 1) / cols);
    const int64_t steps = steps_of(r, products, t.k_step);
    for (int sp = 1; sp <= kMaxSplits; ++sp) {
      const int64_t per = (steps + sp - 1) / sp;
      if (sp > 1 && per * t.k_step < 4 * kBK) break;
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
ProductPlan plan_product(int64_t m, int64_t n, int cols, int64_t r, int products, int words) {
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

Grid grid_of(const Part& part, int64_t m, int64_t k) {
  const LayerPlan& p = part.plan;
  const TileCost& t = kTileCosts[p.tile];
  return Grid{blocks_of(k), (int)((m + t.rows - 1) / t.rows), part.tiles_n, p.steps_per_split, p.splits,
              p.steps_per_split > t.stages - 1 ? p.steps_per_split : t.stages - 1};
}

// One persistent workgroup a CU walks its (tile, split) units.
dim3 blocks_for(const Grid& g) {
  const int64_t units = (int64_t)g.tiles_m * g.tiles_n * g.splits;
  return dim3((uint32_t)(units < device_cus() ? units : device_cus()));
}

// Calls f with the tile as a compile-time constant.
template <int V>
struct Const {
  static constexpr int value = V;
};
template <typename F>
void with_tile(int tile, F&& f) {
  switch (tile) {
    case k256: return f(Const<k256>{});
    case k128: return f(Const<k128>{});
    default: return f(Const<k64>{});
  }
}

// Workspace: split partials of the last part's columns (no other part is
// split; 4096 x 12800 x 5120 backward needs 64 MiB so, and 320 for all columns).
size_t partial_bytes(const ProductPlan& p, int64_t m, int64_t n, int cols, int words) {
  const Part& last = p.part[p.parts - 1];
  const int64_t width = n - (int64_t)last.tile0 * cols;
  return last.plan.splits <= 1
             ? 0
             : round_up((size_t)last.plan.splits * words * partial_slab(m, width) * sizeof(float), kWorkspaceAlign);
}

// Runs a plan: `product(part, grid, partials or null)` launches one part,
// `join(splits, partials, first column)` joins it where it is split.
template <typename Launch, typename Join>
hipError_t run_parts(const ProductPlan& p, int64_t m, int64_t k, int cols, size_t need, void* ws,
                     size_t ws_bytes, Launch&& product, Join&& join) {
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return hipErrorInvalidValue;
  for (int i = 0; i < p.parts; ++i) {
    const Part& part = p.part[i];
    float* const partials = part.plan.splits > 1 ? static_cast<float*>(ws) : nullptr;
    product(part, grid_of(part, m, k), partials);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && partials) e = join(part.plan.splits, partials, (int64_t)part.tile0 * cols);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// Which of a product's two kernels runs: the streams of gemm_layer_skinny.hip
// (up to 32 rows) or the tiles. The streams start and end faster and keep more
// codes in flight; the tiles read X once a workgroup instead of once a wave.
// Measured on MI355X, stream against tiles, microseconds:
//   linear  16 x 25600 x 5120  33.8  38.1    32 x 5120 x 5120   13.3  17.6
//           32 x 8000 x 8192   20.4  22.5    32 x 25600 x 5120  46.4  39.1
//   gated    8 x 25600 x 5120  42.4  51.4    16 x 25600 x 5120  47.5  55.5
//           16 x 5120 x 25600  62.4  51.4    32 x 8192 x 2048   12.4    -
//           32 x 5120 x 5120   21.9  19.9
//   input gradient (rows x weight rows x columns)
//           16 x 12288 x 4096  17.7  21.1    16 x 25600 x 5120  40.5  36
//           32 x 2048 x 4096   10.6  12.2    32 x 5120 x 5120   18.9  16.7
// (Pairs of nine to sixteen rows: past 2^27 codes the stream needs workgroups
// for two a CU, one per 16 columns.)
enum Product { kLinear, kPair, kInputGradient };
bool streams(Product p, int64_t m, int64_t n, int64_t codes) {
  if (m > 32) return false;
  switch (p) {
    case kLinear: return m <= 16 || codes <= (1 << 26);
    case kPair: return m <= 8 || codes <= (m <= 16 ? 1 << 27 : 1 << 25) || (m <= 16 && n >= 8192);
    default: return codes <= (m <= 16 ? 1 << 26 : 1 << 23);
  }
}

size_t linear_act_bytes(int64_t m, int64_t n, int64_t k) {
  if (streams(kLinear, m, n, n * k)) return linear_act_skinny_bytes(m, n, k);
  return partial_bytes(plan_product(m, n, kBN, k, 1, 1), m, n, kBN, 1);
}

hipError_t launch_linear_act(const uint16_t* x, const uint8_t* q, const float* s, uint16_t* y,
                             const LayerEpilogue& ep, int64_t m, int64_t n, int64_t k, void* ws,
                             size_t ws_bytes, hipStream_t stream) {
  if (streams(kLinear, m, n, n * k)) return launch_linear_act_skinny(x, q, s, y, ep, m, n, k, ws, ws_bytes, stream);
  const ProductPlan p = plan_product(m, n, kBN, k, 1, 1);
  return run_parts(
      p, m, k, kBN, partial_bytes(p, m, n, kBN, 1), ws, ws_bytes,
      [&](const Part& part, const Grid& g, float* partials) {
        const LargeArgs la{ep, nullptr, 0, 0, part.tile0};
        const dim3 grid = blocks_for(g);
        with_tile(part.plan.tile, [&](auto tile) {
          constexpr int ID = decltype(tile)::value;
          if (partials) {
            hipLaunchKernelGGL((linear_act_kernel<true, kActNone, ID>), grid, dim3(kThreads), 0, stream, x, q, s,
                               y, partials, (int)m, (int)n, (int)k, g, la);
            return;
          }
          with_act(ep.act, [&](auto a) {
            hipLaunchKernelGGL((linear_act_kernel<false, decltype(a)::value, ID>), grid, dim3(kThreads), 0, stream,
                               x, q, s, y, nullptr, (int)m, (int)n, (int)k, g, la);
          });
        });
      },
      [&](int splits, const float* partials, int64_t c0) {
        return launch_join_layer(partials, y, splits, m, n, c0, ep, stream);
      });
}

size_t glu_bytes(int64_t m, int64_t n, int64_t k) {
  if (streams(kPair, m, n, 2 * n * k)) return glu_skinny_bytes(m, n, k);
  return partial_bytes(plan_product(m, n, kBN / 2, k, 1, 2), m, n, kBN / 2, 2);
}

hipError_t launch_glu(const uint16_t* x, const uint8_t* qg, const float* sg, const uint8_t* qu,
                      const float* su, uint16_t* h, const LayerEpilogue& ep, int64_t m, int64_t n,
                      int64_t k, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (streams(kPair, m, n, 2 * n * k)) return launch_glu_skinny(x, qg, sg, qu, su, h, ep, m, n, k, ws, ws_bytes, stream);
  const ProductPlan p = plan_product(m, n, kBN / 2, k, 1, 2);
  return run_parts(
      p, m, k, kBN / 2, partial_bytes(p, m, n, kBN / 2, 2), ws, ws_bytes,
      [&](const Part& part, const Grid& g, float* partials) {
        const LargeArgs la{ep, nullptr, 0, 0, part.tile0};
        const dim3 grid = blocks_for(g);
        with_tile(part.plan.tile, [&](auto tile) {
          constexpr int ID = decltype(tile)::value;
          if (partials) {
            hipLaunchKernelGGL((glu_kernel<true, kActNone, ID>), grid, dim3(kThreads), 0, stream, x, qg, sg, qu,
                               su, h, partials, (int)m, (int)n, (int)k, g, la);
            return;
          }
          with_act(ep.act, [&](auto a) {
            hipLaunchKernelGGL((glu_kernel<false, decltype(a)::value, ID>), grid, dim3(kThreads), 0, stream, x, qg,
                               sg, qu, su, h, nullptr, (int)m, (int)n, (int)k, g, la);
          });
        });
      },
      [&](int splits, const float* partials, int64_t c0) {
        return launch_join_glu(partials, h, splits, m, n, c0, ep, stream);
      });
}

size_t input_gradient_bytes(int64_t m, int64_t n, int64_t k, int products) {
  if (streams(kInputGradient, m, n, products * n * k)) return input_gradient_skinny_bytes(m, n, k, products);
  return partial_bytes(plan_product(m, k, kBN, n, products, 1), m, k, kBN, 1);
}

hipError_t launch_input_gradient(const uint16_t* a, const uint8_t* q, const float* s, const uint16_t* a2,
                                 const uint8_t* q2, const float* s2, int64_t lda, uint16_t* dx,
                                 int64_t m, int64_t n, int64_t k, void* ws, size_t ws_bytes,
                                 hipStream_t stream) {
  const int products = a2 ? 2 : 1;
  if (streams(kInputGradient, m, n, products * n * k))
    return launch_input_gradient_skinny(a, q, s, a2, q2, s2, lda, dx, m, n, k, ws, ws_bytes, stream);
  const ProductPlan p = plan_product(m, k, kBN, n, products, 1);
  return run_parts(
      p, m, k, kBN, partial_bytes(p, m, k, kBN, 1), ws, ws_bytes,
      [&](const Part& part, const Grid& g, float* partials) {
        const LargeArgs la{LayerEpilogue{}, a2, (int)lda,
                           (int)steps_of(n, 1, kTileCosts[part.plan.tile].k_step), part.tile0};
        const dim3 grid = blocks_for(g);
        with_tile(part.plan.tile, [&](auto tile) {
          constexpr int ID = decltype(tile)::value;
          if (partials)
            hipLaunchKernelGGL((input_gradient_kernel<true, ID>), grid, dim3(kThreads), 0, stream, a, q, s, q2, s2,
                               dx, partials, (int)m, (int)k, (int)n, g, la);
          else
            hipLaunchKernelGGL((input_gradient_kernel<false, ID>), grid, dim3(kThreads), 0, stream, a, q, s, q2,
                               s2, dx, nullptr, (int)m, (int)k, (int)n, g, la);
        });
      },
      [&](int splits, const float* partials, int64_t c0) {
        return launch_join_layer(partials, dx, splits, m, k, c0, LayerEpilogue{}, stream);
      });
}

}  // namespace fp8bl
