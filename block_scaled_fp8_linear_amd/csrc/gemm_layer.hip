// Kernels of the layer operators (fp8bl_layers.h): the epilogues on the
// large-M kernel's loop (gemm_large_body.h) and the input gradient, whose
// reduction runs over the weight's rows.
#include "gemm_large_body.h"

namespace fp8bl {

namespace {

template <int ACT>
__global__ __launch_bounds__(kThreads, 1)
void linear_act_large_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ q,
                             const float* __restrict__ s, uint16_t* __restrict__ y, int M, int N, int K,
                             int gk, int tiles_m, int tiles_n, int steps, LargeArgs la) {
  gemm_large_body<false, false, kLayer, ACT>(x, q, s, nullptr, nullptr, y, nullptr, M, N, K, gk, tiles_m,
                                             tiles_n, steps, 1, max(steps, 2), la);
}

template <int ACT>
__global__ __launch_bounds__(kThreads, 1)
void glu_large_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ qg,
                      const float* __restrict__ sg, const uint8_t* __restrict__ qu,
                      const float* __restrict__ su, uint16_t* __restrict__ h, int M, int N, int K, int gk,
                      int tiles_m, int tiles_n, int steps, LargeArgs la) {
  gemm_large_body<false, false, kGlu, ACT>(x, qg, sg, qu, su, h, nullptr, M, N, K, gk, tiles_m, tiles_n,
                                           steps, 1, max(steps, 2), la);
}

// dx = x W (+ x2 W2): C output columns, R weight rows. The weight's rows are
// the reduction: codes come in as [row][column] and transposing LDS reads
// (ds_read_b64_tr_b8) hand each lane eight rows of its column, so neither a
// transposed copy of the weight nor a shuffle is needed, and one decode per
// code feeds 256 rows as in the forward.
template <bool SPLIT>
__global__ __launch_bounds__(kThreads, 1)
void input_gradient_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ q,
                           const float* __restrict__ s, const uint8_t* __restrict__ q2,
                           const float* __restrict__ s2, uint16_t* __restrict__ dx,
                           float* __restrict__ part, int M, int C, int R, int gk, int tiles_m, int tiles_c,
                           int steps_per_split, int splits, LargeArgs la) {
  gemm_large_body<SPLIT, false, kGradient, kActNone>(x, q, s, q2, s2, dx, part, M, C, R, gk, tiles_m,
                                                     tiles_c, steps_per_split, splits,
                                                     max(steps_per_split, 2), la);
}

int blocks_of(int64_t v) { return (int)((v + kBlock - 1) / kBlock); }

// The input gradient's plan: the large kernel's over the summed reduction.
LargePlan plan_gradient(int64_t m, int64_t n, int64_t k, int products) {
  const int64_t steps = (n + kBK - 1) / kBK * products;
  return plan_large(m, k, steps * kBK);
}

}  // namespace

// Rows up to which the weight-streaming kernels of gemm_layer_skinny.hip run
// (one pass over the weight; they hold two 16-row operands).
constexpr int64_t kSkinnyRows = 32;

size_t linear_act_bytes(int64_t m, int64_t n, int64_t k) {
  return m <= kSkinnyRows ? linear_act_skinny_bytes(m, n, k) : large_workspace_bytes(m, n, k);
}

hipError_t launch_linear_act(const uint16_t* x, const uint8_t* q, const float* s, uint16_t* y,
                             const LayerEpilogue& ep, int64_t m, int64_t n, int64_t k, void* ws,
                             size_t ws_bytes, hipStream_t stream) {
  if (m <= kSkinnyRows) return launch_linear_act_skinny(x, q, s, y, ep, m, n, k, ws, ws_bytes, stream);
  const LargePlan p = plan_large(m, n, k);
  if (p.splits > 1) {
    if (ws == nullptr || ws_bytes < large_workspace_bytes(m, n, k)) return hipErrorInvalidValue;
    float* const part = static_cast<float*>(ws);
    const hipError_t e = launch_gemm_large_partials(p, x, q, s, part, m, n, k, stream);
    if (e != hipSuccess) return e;
    return launch_join_layer(part, y, p.splits, m, n, ep, stream);
  }
  const int tiles_m = (int)((m + kBM - 1) / kBM), tiles_n = (int)((n + kBN - 1) / kBN);
  const int units = tiles_m * tiles_n, grid = units < device_cus() ? units : device_cus();
  const LargeArgs la{ep, nullptr, 0, 0};
  with_act(ep.act, [&](auto a) {
    hipLaunchKernelGGL((linear_act_large_kernel<decltype(a)::value>), dim3((uint32_t)grid), dim3(kThreads), 0,
                       stream, x, q, s, y, (int)m, (int)n, (int)k, blocks_of(k), tiles_m, tiles_n,
                       p.kt_per_split, la);
  });
  return hipGetLastError();
}

size_t glu_bytes(int64_t m, int64_t n, int64_t k) {
  return m <= kSkinnyRows ? glu_skinny_bytes(m, n, k) : 0;
}

hipError_t launch_glu(const uint16_t* x, const uint8_t* qg, const float* sg, const uint8_t* qu,
                      const float* su, uint16_t* h, const LayerEpilogue& ep, int64_t m, int64_t n,
                      int64_t k, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (m <= kSkinnyRows) return launch_glu_skinny(x, qg, sg, qu, su, h, ep, m, n, k, ws, ws_bytes, stream);
  const int tiles_m = (int)((m + kBM - 1) / kBM), tiles_n = (int)((n + kBN / 2 - 1) / (kBN / 2));
  const int units = tiles_m * tiles_n, grid = units < device_cus() ? units : device_cus();
  const LargeArgs la{ep, nullptr, 0, 0};
  with_act(ep.act, [&](auto a) {
    hipLaunchKernelGGL((glu_large_kernel<decltype(a)::value>), dim3((uint32_t)grid), dim3(kThreads), 0, stream,
                       x, qg, sg, qu, su, h, (int)m, (int)n, (int)k, blocks_of(k), tiles_m, tiles_n,
                       (int)((k + kBK - 1) / kBK), la);
  });
  return hipGetLastError();
}

size_t input_gradient_bytes(int64_t m, int64_t n, int64_t k, int products) {
  if (m <= kSkinnyRows) return input_gradient_skinny_bytes(m, n, k, products);
  const LargePlan p = plan_gradient(m, n, k, products);
  if (p.splits <= 1) return 0;
  return round_up((size_t)p.splits * partial_slab(m, k) * sizeof(float), kWorkspaceAlign);
}

hipError_t launch_input_gradient(const uint16_t* a, const uint8_t* q, const float* s, const uint16_t* a2,
                                 const uint8_t* q2, const float* s2, int64_t lda, uint16_t* dx,
                                 int64_t m, int64_t n, int64_t k, void* ws, size_t ws_bytes,
                                 hipStream_t stream) {
  if (m <= kSkinnyRows)
    return launch_input_gradient_skinny(a, q, s, a2, q2, s2, lda, dx, m, n, k, ws, ws_bytes, stream);
  const int products = a2 ? 2 : 1;
  const LargePlan p = plan_gradient(m, n, k, products);
  const int tiles_m = (int)((m + kBM - 1) / kBM), tiles_c = (int)((k + kBN - 1) / kBN);
  const int units = tiles_m * tiles_c * p.splits, grid = units < device_cus() ? units : device_cus();
  LargeArgs la{};
  la.x2 = a2;
  la.ldx = (int)lda;
  la.steps1 = (int)((n + kBK - 1) / kBK);
  if (p.splits == 1) {
    hipLaunchKernelGGL((input_gradient_kernel<false>), dim3((uint32_t)grid), dim3(kThreads), 0, stream, a, q, s,
                       q2, s2, dx, nullptr, (int)m, (int)k, (int)n, blocks_of(k), tiles_m, tiles_c,
                       p.kt_per_split, 1, la);
    return hipGetLastError();
  }
  if (ws == nullptr || ws_bytes < input_gradient_bytes(m, n, k, products)) return hipErrorInvalidValue;
  float* const part = static_cast<float*>(ws);
  hipLaunchKernelGGL((input_gradient_kernel<true>), dim3((uint32_t)grid), dim3(kThreads), 0, stream, a, q, s, q2,
                     s2, dx, part, (int)m, (int)k, (int)n, blocks_of(k), tiles_m, tiles_c, p.kt_per_split,
                     p.splits, la);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_reduce_partials(part, dx, p.splits, m, k, stream);
}

}  // namespace fp8bl
