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
#include "layer_plan.h"

namespace fp8bl {

using namespace plan;

namespace {

static_assert(kTileK == kBK && kTileCols == kBN, "the plans' tiles are the kernels'");

struct Grid {
  int gk, tiles_m, tiles_n, steps, splits, steps_per_unit;
};

// y = act(x W^T + bias) + residual, and z = x W^T + bias where it is saved:
// bias, activation and residual on the fp32 sums in the epilogue, so that z is
// written once and nothing is read back. (8192 x 12288 x 4096 with bias, tanh
// GELU and z saved 672 - 730 us from one card to the next, 1.13 - 1.23 PFLOP/s;
// y alone, plain, 630. 512 x 5120 x 25600 with residual 129 us, 1.04 PFLOP/s;
// 512 x 5120 x 5120 41 us, of which the join of its splits is 7.)
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
