// Row quantizer of the 8-bit integer linear (int8_row.h has the arithmetic),
// bound by its bytes. A row lies in LANES lanes, four chunks of eight values each
// in registers between the maximum and the codes, so x is read once: 16 lanes
// up to K = 512, a wave to 2048, 256 threads to 8192 and 1024 to 32768. A longer
// row is read twice by 1024 threads.
//
// MI355X, against one workgroup of 256 a row that reads it twice: 16384 x 8192
// bf16 74 us (5.4 TB/s) against 90, 25600 x 5120 fp32 119 against 147, 100000 x
// 64 10.3 against 62, 4 x 131056 16 against 35.
#include "fp8bl_ops.h"
#include "int8_row.h"

namespace fp8bl {

namespace {

constexpr int kChunks = 4;                                        // of eight values, in a lane's registers
constexpr int64_t kWorkgroups = (int64_t)1 << 21;                 // of a launch, which has fewer than 2^32 threads

// Maximum over the LANES lanes of a row, in each of them.
template <int LANES>
__device__ __forceinline__ float row_max(float v, float* wave_max) {
  constexpr int kIn = LANES < 64 ? LANES : 64;
#pragma unroll
  for (int off = kIn / 2; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  if constexpr (LANES > 64) {
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = v;
    __syncthreads();
    v = wave_max[0];
#pragma unroll
    for (int w = 1; w < LANES / 64; ++w) v = fmaxf(v, wave_max[w]);
  }
  return v;
}

template <int LANES, bool LONG, typename T>
__global__ __launch_bounds__(LANES > 256 ? LANES : 256)
void int8_quantize_kernel(const T* __restrict__ x, int8_t* __restrict__ q, float* __restrict__ scale, int M, int K) {
  constexpr int kThreads = LANES > 256 ? LANES : 256, kRows = kThreads / LANES;
  __shared__ float wave_max[LANES > 64 ? LANES / 64 : 1];
  const int lane = threadIdx.x % LANES;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / LANES;
  const bool live = row < M;                 // for all of a workgroup where a row takes more than a wave
  const T* const xr = x + (live ? row : 0) * K;
  int8_t* const qr = q + (live ? row : 0) * K;
  float v[kChunks][8];
  float amax = 0.0f;
  if constexpr (LONG) {
    for (int c = lane * 8; c < K; c += LANES * 8) {
      load8(xr + c, v[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[0][i]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = (lane + LANES * j) * 8;
      if (live && c < K)
        load8(xr + c, v[j]);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[j][i]));
  }
  const RowScale r = int8_scale(row_max<LANES>(amax, wave_max));
  if (!live) return;
  if (lane == 0) scale[row] = r.s;
  if constexpr (LONG) {
    for (int c = lane * 8; c < K; c += LANES * 8) {
      load8(xr + c, v[0]);
      *reinterpret_cast<u32x2*>(qr + c) = codes8(v[0], r);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = (lane + LANES * j) * 8;
      if (c >= K) break;
      *reinterpret_cast<u32x2*>(qr + c) = codes8(v[j], r);
    }
  }
}

template <int LANES, bool LONG, typename T>
hipError_t launch(const T* x, int8_t* q, float* scale, int64_t m, int64_t k, hipStream_t stream) {
  constexpr int kThreads = LANES > 256 ? LANES : 256, kRows = kThreads / LANES;
  for (int64_t r = 0; r < m; r += kWorkgroups * kRows) {
    const int64_t rows = m - r < kWorkgroups * kRows ? m - r : kWorkgroups * kRows;
    hipLaunchKernelGGL((int8_quantize_kernel<LANES, LONG, T>), dim3((uint32_t)((rows + kRows - 1) / kRows)),
                       dim3(kThreads), 0, stream, x + r * k, q + r * k, scale + r, (int)rows, (int)k);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T>
hipError_t launch_any(const T* x, int8_t* q, float* scale, int64_t m, int64_t k, hipStream_t stream) {
  constexpr int64_t kEach = 8 * kChunks;
  return k <= 16 * kEach     ? launch<16, false>(x, q, scale, m, k, stream)
         : k <= 64 * kEach   ? launch<64, false>(x, q, scale, m, k, stream)
         : k <= 256 * kEach  ? launch<256, false>(x, q, scale, m, k, stream)
         : k <= 1024 * kEach ? launch<1024, false>(x, q, scale, m, k, stream)
                             : launch<1024, true>(x, q, scale, m, k, stream);
}

}  // namespace

hipError_t launch_int8_quantize(const float* x, int8_t* q, float* scale, int64_t m, int64_t k, hipStream_t stream) {
  return launch_any(x, q, scale, m, k, stream);
}
hipError_t launch_int8_quantize(const uint16_t* x, int8_t* q, float* scale, int64_t m, int64_t k,
                                hipStream_t stream) {
  return launch_any(x, q, scale, m, k, stream);
}

}  // namespace fp8bl
