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

// Joins split partials and applies the linear's epilogue: the partials added
// in split order, then bias, activation, residual and one rounding each of z
// and y. VEC outputs a thread (8 where N is a multiple of 8: then they lie in
// one row), grid-stride.
template <int ACT, int VEC>
__global__ __launch_bounds__(256)
void reduce_layer_kernel(const float* __restrict__ part, uint16_t* y, int splits, size_t mn, size_t slab,
                         uint32_t n, LayerEpilogue ep) {
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * VEC; i < mn;
       i += (size_t)gridDim.x * 256 * VEC) {
    float t[VEC];
    if constexpr (VEC == 8) {
      f32x4 a = *reinterpret_cast<const f32x4*>(part + i);
      f32x4 b = *reinterpret_cast<const f32x4*>(part + i + 4);
#pragma unroll 4
      for (int sp = 1; sp < splits; ++sp) {
        const f32x4 c = *reinterpret_cast<const f32x4*>(part + (size_t)sp * slab + i);
        const f32x4 d = *reinterpret_cast<const f32x4*>(part + (size_t)sp * slab + i + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[e] += c[e];
          b[e] += d[e];
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        t[e] = a[e];
        t[4 + e] = b[e];
      }
    } else {
      t[0] = part[i];
      for (int sp = 1; sp < splits; ++sp) t[0] += part[(size_t)sp * slab + i];
    }
    const uint32_t col = (uint32_t)(i % n);
    uint32_t zo[VEC], yo[VEC], bias[VEC], res[VEC];
    if constexpr (VEC == 8) {
      u32x4 bv = {}, rv = {};
      if (ep.bias) bv = *reinterpret_cast<const u32x4*>(ep.bias + col);
      if (ep.residual) rv = *reinterpret_cast<const u32x4*>(ep.residual + i);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        bias[e] = (e & 1) ? bv[e >> 1] & 0xFFFF0000u : bv[e >> 1] << 16;
        res[e] = (e & 1) ? rv[e >> 1] & 0xFFFF0000u : rv[e >> 1] << 16;
      }
    } else {
      bias[0] = ep.bias ? (uint32_t)ep.bias[col] << 16 : 0;
      res[0] = ep.residual ? (uint32_t)ep.residual[i] << 16 : 0;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float z = t[e] + __uint_as_float(bias[e]);
      float v = act_f32<ACT>(z);
      if (ep.residual) v += __uint_as_float(res[e]);
      zo[e] = f32_bf16(z);
      yo[e] = f32_bf16(v);
    }
    if constexpr (VEC == 8) {
      const u32x4 zv = {zo[0] | zo[1] << 16, zo[2] | zo[3] << 16, zo[4] | zo[5] << 16, zo[6] | zo[7] << 16};
      const u32x4 yv = {yo[0] | yo[1] << 16, yo[2] | yo[3] << 16, yo[4] | yo[5] << 16, yo[6] | yo[7] << 16};
      if (ep.z) *reinterpret_cast<u32x4*>(ep.z + i) = zv;
      *reinterpret_cast<u32x4*>(y + i) = yv;
    } else {
      if (ep.z) ep.z[i] = (uint16_t)zo[0];
      y[i] = (uint16_t)yo[0];
    }
  }
}

hipError_t launch_reduce_layer(const float* part, uint16_t* y, int splits, int64_t m, int64_t n,
                               const LayerEpilogue& ep, hipStream_t stream) {
  const size_t mn = (size_t)m * n, slab = partial_slab(m, n);
  const bool wide = n % 8 == 0;
  const size_t blocks = (mn + (wide ? 2047 : 255)) / (wide ? 2048 : 256);
  const dim3 grid((uint32_t)(blocks < (1u << 20) ? blocks : (1u << 20)));
  with_act(ep.act, [&](auto a) {
    constexpr int A = decltype(a)::value;
    if (wide)
      hipLaunchKernelGGL((reduce_layer_kernel<A, 8>), grid, dim3(256), 0, stream, part, y, splits, mn, slab,
                         (uint32_t)n, ep);
    else
      hipLaunchKernelGGL((reduce_layer_kernel<A, 1>), grid, dim3(256), 0, stream, part, y, splits, mn, slab,
                         (uint32_t)n, ep);
  });
  return hipGetLastError();
}

int blocks_of(int64_t v) { return (int)((v + kBlock - 1) / kBlock); }

// The input gradient's plan: the large kernel's over the summed reduction.
LargePlan plan_gradient(int64_t m, int64_t n, int64_t k, int products) {
  const int64_t steps = (n + kBK - 1) / kBK * products;
  return plan_large(m, k, steps * kBK);
}

}  // namespace

size_t linear_act_bytes(int64_t m, int64_t n, int64_t k) { return large_workspace_bytes(m, n, k); }

hipError_t launch_linear_act(const uint16_t* x, const uint8_t* q, const float* s, uint16_t* y,
                             const LayerEpilogue& ep, int64_t m, int64_t n, int64_t k, void* ws,
                             size_t ws_bytes, hipStream_t stream) {
  const LargePlan p = plan_large(m, n, k);
  if (p.splits > 1) {
    if (ws == nullptr || ws_bytes < large_workspace_bytes(m, n, k)) return hipErrorInvalidValue;
    float* const part = static_cast<float*>(ws);
    const hipError_t e = launch_gemm_large_partials(p, x, q, s, part, m, n, k, stream);
    if (e != hipSuccess) return e;
    return launch_reduce_layer(part, y, p.splits, m, n, ep, stream);
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

size_t glu_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_glu(const uint16_t* x, const uint8_t* qg, const float* sg, const uint8_t* qu,
                      const float* su, uint16_t* h, const LayerEpilogue& ep, int64_t m, int64_t n,
                      int64_t k, void*, size_t, hipStream_t stream) {
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
  const LargePlan p = plan_gradient(m, n, k, products);
  if (p.splits <= 1) return 0;
  return round_up((size_t)p.splits * partial_slab(m, k) * sizeof(float), kWorkspaceAlign);
}

hipError_t launch_input_gradient(const uint16_t* a, const uint8_t* q, const float* s, const uint16_t* a2,
                                 const uint8_t* q2, const float* s2, int64_t lda, uint16_t* dx,
                                 int64_t m, int64_t n, int64_t k, void* ws, size_t ws_bytes,
                                 hipStream_t stream) {
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
