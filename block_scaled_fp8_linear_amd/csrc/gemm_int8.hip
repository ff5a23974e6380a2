// 8-bit integer GEMM:
//   Y[m,n] = bf16( float(sum_k xq[m,k] wq[n,k]) * (xs[m] * ws[n]) + bias[n] )
// with the sum exact in int32 (v_mfma_i32_16x16x64_i8).
//
// v_mfma_i32_16x16x64_i8: lane l supplies 16 consecutive-k codes of row
// l % 16 of its block at k chunk l / 16, for A and B alike. The weight is the A
// operand and X the B operand, so a lane's four sums are rows 4 (l / 16) .. +3
// of the weight block, four consecutive output columns of X row l % 16.
#include "fp8bl_device.h"
#include "fp8bl_ops.h"

namespace fp8bl {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

// 64 x 64 outputs a workgroup, 64 rows of X by 16 columns a wave, operands
// straight from memory.
__global__ __launch_bounds__(kThreads)
void gemm_int8_kernel(const int8_t* __restrict__ xq, const float* __restrict__ xs, const int8_t* __restrict__ wq,
                      const float* __restrict__ ws, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y,
                      int M, int N, int K, int tiles_n) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * 64;
  const int n0 = (int)(blockIdx.x % tiles_n) * 64 + 16 * wave;
  const int r = lane & 15, g = lane >> 4;
  i32x4 acc[4] = {};
  for (int k0 = 0; k0 < K; k0 += 64) {
    const int c = k0 + 16 * g;
    i32x4 a = {}, b[4] = {};
    if (c < K) {
      if (n0 + r < N) a = *reinterpret_cast<const i32x4*>(wq + (size_t)(n0 + r) * K + c);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (m0 + 16 * i + r < M) b[i] = *reinterpret_cast<const i32x4*>(xq + (size_t)(m0 + 16 * i + r) * K + c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b[i], acc[i], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = m0 + 16 * i + r;
    if (row >= M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = n0 + 4 * g + j;
      if (col >= N) continue;
      float v = (float)acc[i][j] * (xs[row] * ws[col]);
      if (bias) v += bf16_f32(bias[col]);
      y[(size_t)row * N + col] = f32_bf16(v);
    }
  }
}

}  // namespace

size_t int8_gemm_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_int8_gemm(const int8_t* xq, const float* xs, const int8_t* wq, const float* ws,
                            const uint16_t* bias, uint16_t* y, int64_t m, int64_t n, int64_t k, void*,
                            hipStream_t stream) {
  const int64_t tiles_n = (n + 63) / 64;
  const int64_t rows = 64 * (((int64_t)1 << 23) / tiles_n);   // a launch has fewer than 2^32 threads
  for (int64_t r0 = 0; r0 < m; r0 += rows) {
    const int64_t mr = m - r0 < rows ? m - r0 : rows;
    hipLaunchKernelGGL(gemm_int8_kernel, dim3((uint32_t)((mr + 63) / 64 * tiles_n)), dim3(kThreads), 0, stream,
                       xq + (size_t)r0 * k, xs + r0, wq, ws, bias, y + (size_t)r0 * n, (int)mr, (int)n, (int)k,
                       (int)tiles_n);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp8bl
