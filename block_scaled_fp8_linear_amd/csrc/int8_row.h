// Quantization of a row to 8-bit integers:
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

}  // namespace

}  // namespace fp8bl
