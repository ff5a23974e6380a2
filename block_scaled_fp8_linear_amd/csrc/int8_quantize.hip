// Row quantizer of the 8-bit integer linear (int8_row.h has the arithmetic): one
// workgroup a row.
#include "fp8bl_ops.h"
#include "int8_row.h"

namespace fp8bl {

namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ __launch_bounds__(kThreads)
void int8_quantize_kernel(const T* __restrict__ x, int8_t* __restrict__ q, float* __restrict__ scale, int K) {
  __shared__ float wave_max[kThreads / 64];
  const size_t row = blockIdx.x;
  const float s = int8_quantize_row<kThreads>(x + row * K, q + row * K, K, wave_max);
  if (threadIdx.x == 0) scale[row] = s;
}

template <typename T>
hipError_t launch(const T* x, int8_t* q, float* scale, int64_t m, int64_t k, hipStream_t stream) {
  constexpr int64_t kRows = (int64_t)1 << 22;     // of a launch, which has fewer than 2^32 threads
  for (int64_t r = 0; r < m; r += kRows) {
    hipLaunchKernelGGL(int8_quantize_kernel<T>, dim3((uint32_t)(m - r < kRows ? m - r : kRows)), dim3(kThreads), 0,
                       stream, x + r * k, q + r * k, scale + r, (int)k);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_int8_quantize(const float* x, int8_t* q, float* scale, int64_t m, int64_t k, hipStream_t stream) {
  return launch(x, q, scale, m, k, stream);
}
hipError_t launch_int8_quantize(const uint16_t* x, int8_t* q, float* scale, int64_t m, int64_t k,
                                hipStream_t stream) {
  return launch(x, q, scale, m, k, stream);
}

}  // namespace fp8bl
