// Argument checks shared by the ABI files (host only, no HIP calls).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "fp8bl.h"

#define FP8BL_EXPORT extern "C" __attribute__((visibility("default")))

namespace fp8bl {
namespace checks {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxDim = (int64_t)1 << 31;     // every dimension fits int32
constexpr int64_t kMaxElems = (int64_t)1 << 35;   // N*K, M*K and M*N stay below this (8-element chunk index fits uint32)

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

inline size_t grid_elems(int64_t n, int64_t k) {
  return (size_t)((n + FP8BL_BLOCK - 1) / FP8BL_BLOCK) * (size_t)((k + FP8BL_BLOCK - 1) / FP8BL_BLOCK);
}

inline int check_nk(int64_t n, int64_t k) {
  if (n < 0 || k <= 0 || (k % 16) != 0) return FP8BL_INVALID_ARG;
  if (n >= kMaxDim || k >= kMaxDim || (n > 0 && n * k >= kMaxElems)) return FP8BL_INVALID_ARG;
  if ((n + FP8BL_BLOCK - 1) / FP8BL_BLOCK > 65535) return FP8BL_INVALID_ARG;
  return FP8BL_OK;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? FP8BL_OK : FP8BL_HIP_ERROR; }

}  // namespace checks
}  // namespace fp8bl
