// The layer operators' products, in their simplest right form: a 64x64 tile
// of fp32 sums per workgroup, operands decoded into LDS 16 of the reduction
// at a time, 16 FMAs a thread and step. Takes every shape.
#include "fp8bl_act.h"
#include "fp8bl_device.h"
#include "fp8bl_internal.h"

namespace fp8bl {

namespace {

constexpr int kT = 64, kR = 16;

__device__ __forceinline__ float bf16_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t f32_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

__device__ float act_any(int act, float t) {
  switch (act) {
    case kActRelu: return act_f32<kActRelu>(t);
    case kActSilu: return act_f32<kActSilu>(t);
    case kActGelu: return act_f32<kActGelu>(t);
    case kActGeluTanh: return act_f32<kActGeluTanh>(t);
    default: return t;
  }
}

struct SimpleArgs {
  const uint16_t* a[2];    // [M, R] rows of lda
  const uint8_t* q[2];     // weights, [cols, R] or (TRANS) [R, cols]
  const float* s[2];
  int64_t lda;
  int64_t M, C, R;         // rows, output columns, reduction
  int gk;                  // scale grid columns
  LayerEpilogue ep;
};

// MODE 0: y = act(z) + residual. MODE 1: the gated pair. MODE 2: the sum of
// the two products (or the first), rounded.
template <bool TRANS, int MODE>
__global__ __launch_bounds__(256)
void gemm_simple_kernel(SimpleArgs P, uint16_t* __restrict__ y, int tiles_c) {
  __shared__ float as[kR][kT + 1], bs[kR][kT + 1];
  const int64_t m0 = (int64_t)(blockIdx.x / (uint32_t)tiles_c) * kT;
  const int64_t c0 = (int64_t)(blockIdx.x % (uint32_t)tiles_c) * kT;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[2][4][4] = {};
  for (int p = 0; p < 2; ++p) {
    if (!P.q[p]) break;
    for (int64_t r0 = 0; r0 < P.R; r0 += kR) {
      for (int i = threadIdx.x; i < kT * kR; i += 256) {
        const int row = i / kR, r = i % kR;
        const bool in = m0 + row < P.M && r0 + r < P.R;
        as[r][row] = in ? bf16_f32(P.a[p][(m0 + row) * P.lda + r0 + r]) : 0.0f;
        const int bc = TRANS ? i % kT : i / kR, br = TRANS ? i / kT : i % kR;
        float w = 0.0f;
        if (c0 + bc < P.C && r0 + br < P.R) {
          const int64_t n = TRANS ? r0 + br : c0 + bc, k = TRANS ? c0 + bc : r0 + br;
          const uint8_t code = P.q[p][n * (TRANS ? P.C : P.R) + k];
          const f32x2 v = __builtin_amdgcn_cvt_pk_f32_fp8((int)code, false);
          w = (float)(__bf16)__fmul_rn(v[0], P.s[p][(n / kBlock) * P.gk + k / kBlock]);
        }
        bs[br][bc] = w;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float& t = acc[MODE == 1 ? p : 0][i][j];
            t = fmaf(as[r][ty * 4 + i], bs[r][tx + 16 * j], t);
          }
      __syncthreads();
    }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t row = m0 + ty * 4 + i, col = c0 + tx + 16 * j;
      if (row >= P.M || col >= P.C) continue;
      const int64_t at = row * P.C + col;
      float v = acc[0][i][j];
      if (MODE == 0) {
        if (P.ep.bias) v += bf16_f32(P.ep.bias[col]);
        if (P.ep.z) P.ep.z[at] = f32_bf16(v);
        v = act_any(P.ep.act, v);
        if (P.ep.residual) v += bf16_f32(P.ep.residual[at]);
      }
      if (MODE == 1) {
        const float u = acc[1][i][j];
        if (P.ep.g) P.ep.g[at] = f32_bf16(v);
        if (P.ep.u) P.ep.u[at] = f32_bf16(u);
        v = act_any(P.ep.act, v) * u;
      }
      y[at] = f32_bf16(v);
    }
}

template <bool TRANS, int MODE>
hipError_t launch(const SimpleArgs& P, uint16_t* y, hipStream_t stream) {
  const int64_t tc = (P.C + kT - 1) / kT, tm = (P.M + kT - 1) / kT;
  if (tc * tm >= (1 << 24)) return hipErrorInvalidValue;
  hipLaunchKernelGGL((gemm_simple_kernel<TRANS, MODE>), dim3((uint32_t)(tc * tm)), dim3(256), 0, stream,
                     P, y, (int)tc);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_act(const uint16_t* x, const uint8_t* q, const float* s, uint16_t* y,
                             const LayerEpilogue& ep, int64_t m, int64_t n, int64_t k, void*, size_t,
                             hipStream_t stream) {
  const SimpleArgs P{{x, nullptr}, {q, nullptr}, {s, nullptr}, k, m, n, k, (int)((k + kBlock - 1) / kBlock), ep};
  return launch<false, 0>(P, y, stream);
}

hipError_t launch_glu(const uint16_t* x, const uint8_t* qg, const float* sg, const uint8_t* qu,
                      const float* su, uint16_t* h, const LayerEpilogue& ep, int64_t m, int64_t n,
                      int64_t k, void*, size_t, hipStream_t stream) {
  const SimpleArgs P{{x, x}, {qg, qu}, {sg, su}, k, m, n, k, (int)((k + kBlock - 1) / kBlock), ep};
  return launch<false, 1>(P, h, stream);
}

hipError_t launch_input_gradient(const uint16_t* a, const uint8_t* q, const float* s, const uint16_t* a2,
                                 const uint8_t* q2, const float* s2, int64_t lda, uint16_t* dx,
                                 int64_t m, int64_t n, int64_t k, void*, size_t, hipStream_t stream) {
  const SimpleArgs P{{a, a2}, {q, q2}, {s, s2}, lda, m, k, n, (int)((k + kBlock - 1) / kBlock), {}};
  return launch<true, 2>(P, dx, stream);
}

size_t linear_act_bytes(int64_t, int64_t, int64_t) { return 0; }
size_t glu_bytes(int64_t, int64_t, int64_t) { return 0; }
size_t input_gradient_bytes(int64_t, int64_t, int64_t, int) { return 0; }

}  // namespace fp8bl
