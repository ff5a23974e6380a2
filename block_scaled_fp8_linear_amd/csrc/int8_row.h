// Quantization of one row to 8-bit integers by a workgroup:
//   S = fl32(max |x| / 127), 1 where that is 0;
//   code = the integer nearest to fl32(x / S), ties to even, within +-127.
#pragma once

#include "fp8bl_device.h"

namespace fp8bl {

namespace {

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

// The scale of a row and what its codes are worked out with.
struct RowScale {
  float s, inv;
  bool plain;       // subnormal scales and their like: every code by IEEE division
};

// fl32(v / s) to the nearest integer, ties to even, within +-127, packed.
//
// v inv is off from the quotient by at most 127 2^-23 (two roundings), so its
// nearest integer is the quotient's unless it lies within 2^-15 of a half: then
// the eight are taken by IEEE division (0.05% of them).
constexpr float kRound = 12582912.0f;      // 1.5 2^23: a sum with it has the nearest integer in its low bits

__device__ __forceinline__ u32x2 pack_codes(const float (&t)[8]) {
  auto pack4 = [&](int i) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[i + 1]), __float_as_uint(t[i]), 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[i + 3]), __float_as_uint(t[i + 2]), 0x04000C0Cu);
    return lo | hi;
  };
  return u32x2{pack4(0), pack4(4)};
}
__device__ __forceinline__ u32x2 codes8(const float (&v)[8], const RowScale& r) {
  float t[8], off = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = v[i] * r.inv;
    t[i] = q + kRound;
    off = fmaxf(off, fabsf(q - (t[i] - kRound)));
  }
  if (r.plain || off > 0.5f - 0x1p-15f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = fminf(fmaxf(__fdiv_rn(v[i], r.s), -127.0f), 127.0f) + kRound;
  }
  return pack_codes(t);
}

__device__ __forceinline__ RowScale int8_scale(float amax) {
  float s = __fdiv_rn(amax, 127.0f);
  if (s == 0.0f) s = 1.0f;
  return RowScale{s, __fdiv_rn(1.0f, s), s < 0x1p-100f};
}

// One row by a workgroup of THREADS: the maximum in a first pass, the codes in a
// second, which finds the row in the cache. Returns the scale, in every thread.
// `wave_max` holds one float a wave.
template <int THREADS, typename T>
__device__ __forceinline__ float int8_quantize_row(const T* __restrict__ x, int8_t* q, int K, float* wave_max) {
  float amax = 0.0f;
  for (int c = threadIdx.x * 8; c < K; c += THREADS * 8) {
    float v[8];
    load8(x + c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
  __syncthreads();           // the last row's maxima have been read
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = amax;
  __syncthreads();
  amax = wave_max[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) amax = fmaxf(amax, wave_max[w]);
  const RowScale r = int8_scale(amax);
  for (int c = threadIdx.x * 8; c < K; c += THREADS * 8) {
    float v[8];
    load8(x + c, v);
    *reinterpret_cast<u32x2*>(q + c) = codes8(v, r);
  }
  return r.s;
}

}  // namespace

}  // namespace fp8bl
