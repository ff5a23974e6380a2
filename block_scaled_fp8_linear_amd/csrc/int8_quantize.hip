// Row quantizer of the 8-bit integer linear: for each row of x[M,K],
//   S = fl32(max |x| / 127), 1 where that is 0;
//   code = the integer nearest to fl32(x / S), ties to even, within +-127.
// (S can be a subnormal of few bits, whose quotients pass 127; it is 0 for an
// fp32 row below 2^-143.) One workgroup a row: the maximum in a first pass, the
// codes in a second, which finds the row in the cache.
#include "fp8bl_device.h"
#include "fp8bl_ops.h"

namespace fp8bl {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(a[i] << 16);
    v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads)
void int8_quantize_kernel(const T* __restrict__ x, int8_t* __restrict__ q, float* __restrict__ scale, int K) {
  __shared__ float wave_max[kThreads / 64];
  const size_t row = blockIdx.x;
  const T* const xr = x + row * K;
  float amax = 0.0f;
  for (int c = threadIdx.x * 8; c < K; c += kThreads * 8) {
    float v[8];
    load8(xr + c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(wave_max[0], wave_max[1]), fmaxf(wave_max[2], wave_max[3]));
  float s = __fdiv_rn(amax, 127.0f);
  if (s == 0.0f) s = 1.0f;
  if (threadIdx.x == 0) scale[row] = s;
  for (int c = threadIdx.x * 8; c < K; c += kThreads * 8) {
    float v[8];
    load8(xr + c, v);
    u32x2 out = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = fminf(fmaxf(rintf(__fdiv_rn(v[i], s)), -127.0f), 127.0f);
      out[i >> 2] |= ((uint32_t)(int)t & 0xFFu) << (8 * (i & 3));
    }
    *reinterpret_cast<u32x2*>(q + row * K + c) = out;
  }
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
