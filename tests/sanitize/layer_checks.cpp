// Host-side argument checks of the layer operators' C ABI under
// AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_layers_sanitize_cpu.py): extreme sizes, activations and
// pointers, none dereferenced; every call returns from validation.
#include <cstdint>
#include <cstdio>

#include <hip/hip_runtime.h>

#include "fp8bl_layers.h"

namespace {
template <typename T>
T* at(uintptr_t i) { return reinterpret_cast<T*>(i << 44); }
}  // namespace

int main() {
  int devices = 0;
  if (hipGetDeviceCount(&devices) == hipSuccess && devices > 0) {
    std::printf("SKIP: a HIP device is present\n");
    return 0;
  }
  int fail = 0;
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 8, 15, 16, 17, 128, 1003, (int64_t)1 << 20, ((int64_t)1 << 20) + 16,
                           ((int64_t)1 << 31) - 1, (int64_t)1 << 31, (int64_t)1 << 35, INT64_MAX};
  const int acts[] = {-1, 0, 1, 4, 5, INT32_MAX};
  uint16_t *a = at<uint16_t>(1), *b = at<uint16_t>(2), *c = at<uint16_t>(3), *d = at<uint16_t>(4),
           *e = at<uint16_t>(5), *f = at<uint16_t>(6);
  uint8_t *q = at<uint8_t>(7), *q2 = at<uint8_t>(8);
  float *s = at<float>(9), *s2 = at<float>(10), *db = at<float>(11);
  void* ws = at<void>(12);
  const size_t wb = (size_t)1 << 43;
  for (int64_t m : sizes)
    for (int64_t n : sizes)
      for (int64_t k : sizes) {
        const size_t need[] = {fp8_block_linear_act_workspace_size(m, n, k),
                               fp8_block_linear_act_backward_workspace_size(m, n, k),
                               fp8_block_glu_workspace_size(m, n, k), fp8_block_glu_backward_workspace_size(m, n, k)};
        for (size_t v : need)
          if (v % 256 != 0) {
            std::printf("FAIL workspace m=%lld n=%lld k=%lld\n", (long long)m, (long long)n, (long long)k);
            ++fail;
          }
        for (int act : acts) {
          const bool none = act == 0;
          const int st[] = {
              fp8_block_linear_act(a, q, s, b, c, d, e, m, n, k, act, ws, wb, nullptr),
              fp8_block_linear_act_backward(a, none ? nullptr : b, q, s, none ? nullptr : c, db, d, m, n, k, act, ws,
                                            wb, nullptr),
              fp8_block_glu(a, q, s, q2, s2, b, c, d, m, n, k, act, ws, wb, nullptr),
              fp8_block_glu_backward(a, b, c, q, s, q2, s2, d, e, f, m, n, k, act, ws, wb, nullptr),
              fp8_block_linear_act(a, q, s, b, c, d, e, m, n, k, act, nullptr, 0, nullptr),
              fp8_block_glu(nullptr, q, s, q2, s2, b, c, d, m, n, k, act, ws, wb, nullptr)};
          for (int v : st)
            if (v == FP8BL_OK && m != 0 && n != 0) {
              std::printf("FAIL accepted m=%lld n=%lld k=%lld act=%d\n", (long long)m, (long long)n, (long long)k, act);
              ++fail;
            }
          if ((act < 0 || act > 4) && st[0] != FP8BL_INVALID_ARG) ++fail;
        }
      }
  std::printf("%s: %d failures\n", fail ? "FAILED" : "OK", fail);
  return fail ? 1 : 0;
}
