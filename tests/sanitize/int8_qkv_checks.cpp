// Host-side argument checks of include/fp8bl_int8.h and include/fp8bl_qkv.h under
// AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_int8_qkv_sanitize_cpu.py): extreme sizes, strides and pointers,
// none dereferenced but the argument structure; every call returns from
// validation.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>

#include <hip/hip_runtime.h>

#include "fp8bl_int8.h"
#include "fp8bl_qkv.h"

namespace {
template <typename T>
T* at(uintptr_t i) { return reinterpret_cast<T*>(i << 44); }

int fail = 0;
void expect(bool ok, const char* what, int64_t a, int64_t b, int64_t c) {
  if (!ok) {
    std::printf("FAIL %s %lld %lld %lld\n", what, (long long)a, (long long)b, (long long)c);
    ++fail;
  }
}
bool refused(int st) { return st != FP8BL_OK; }
}  // namespace

int main() {
  int devices = 0;
  if (hipGetDeviceCount(&devices) == hipSuccess && devices > 0) {
    std::printf("SKIP: a HIP device is present\n");
    return 0;
  }
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 8, 15, 16, 17, 128, 1003, 4096, 4097, 65536, 65537, 131056, 131072,
                           (int64_t)1 << 20, ((int64_t)1 << 20) + 16, ((int64_t)1 << 31) - 1, (int64_t)1 << 31,
                           (int64_t)1 << 35, INT64_MAX};
  const size_t wb = (size_t)1 << 43;
  for (int64_t m : sizes)
    for (int64_t k : sizes) {
      const int a = int8_row_quantize(at<float>(1), at<int8_t>(2), at<float>(3), m, k, nullptr);
      const int b = int8_row_quantize_bf16(at<uint16_t>(1), at<int8_t>(2), at<float>(3), m, k, nullptr);
      expect(m == 0 || (refused(a) && refused(b)), "quantize", m, k, 0);
      for (int64_t n : sizes) {
        const size_t w0 = int8_linear_workspace_size(m, n, k), w1 = int8_linear_bf16_workspace_size(m, n, k);
        expect(w0 % 256 == 0 && w1 % 256 == 0 && w1 >= w0, "workspace", m, n, k);
        const int c = int8_linear(at<int8_t>(1), at<float>(2), at<int8_t>(3), at<float>(4), at<uint16_t>(5),
                                  at<uint16_t>(6), m, n, k, at<void>(7), wb, nullptr);
        const int d = int8_linear_bf16(at<uint16_t>(1), at<int8_t>(3), at<float>(4), nullptr, at<uint16_t>(6), m, n, k,
                                       at<void>(7), wb, nullptr);
        expect(m == 0 || n == 0 || (refused(c) && refused(d)), "linear", m, n, k);
        expect(refused(int8_linear(nullptr, at<float>(2), at<int8_t>(3), at<float>(4), nullptr, at<uint16_t>(6), m, n, k,
                                   nullptr, 0, nullptr)) || m == 0 || n == 0, "null", m, n, k);
      }
    }

  const double eps[] = {0.0, 1e-6, -1.0, std::numeric_limits<double>::quiet_NaN(), std::numeric_limits<double>::infinity(),
                        1e300};
  auto all = [&](const fp8bl_qkv& g) {
    const int st[] = {fp8_qk_norm_rope(&g, nullptr), fp8_qk_norm_rope_backward(&g, at<void>(90), wb, nullptr),
                      fp8_kv_store(&g, nullptr), fp8_kv_load(&g, nullptr), fp8_qk_norm_rope_store(&g, nullptr)};
    (void)fp8_qk_norm_rope_backward_workspace_size(g.tokens, g.q_heads, g.k_heads, g.head_dim);
    if (g.tokens > 0 && g.q_heads > 0 && g.k_heads > 0)
      for (int s : st) expect(refused(s), "accepted", g.tokens, g.q_heads, g.head_dim);
  };
  fp8bl_qkv base{};
  base.tokens = 4, base.q_heads = 6, base.k_heads = 2, base.head_dim = 32;
  fp8bl_heads* views[] = {&base.q, &base.k, &base.v, &base.q_out, &base.k_out, &base.v_out, &base.dq, &base.dk};
  for (int i = 0; i < 8; ++i) *views[i] = fp8bl_heads{at<uint16_t>(10 + i), 6 * 32, 32};
  base.q_weight = at<uint16_t>(20), base.k_weight = at<uint16_t>(21);
  base.dq_weight = at<float>(22), base.dk_weight = at<float>(23);
  base.positions = at<int32_t>(24), base.inv_freq = at<float>(25);
  base.axes = 1, base.pairs = 16, base.eps = 1e-6;
  base.slots = at<int32_t>(26), base.k_cache = at<uint8_t>(30), base.v_cache = at<uint8_t>(40);
  base.k_scale = at<float>(50), base.v_scale = at<float>(60), base.cache_rows = 10;
  for (int64_t a : sizes)
    for (int64_t b : sizes)
      for (int which = 0; which < 10; ++which) {
        fp8bl_qkv g = base;
        int64_t* members[] = {&g.tokens, &g.q_heads, &g.k_heads, &g.head_dim, &g.axes, &g.pairs, &g.interleaved,
                              &g.cache_rows, &g.q.token_stride, &g.k_out.head_stride};
        *members[which] = a;
        *members[(which + 3) % 10] = b;
        all(g);
      }
  for (double e : eps)
    for (int64_t s : sizes)
      for (int64_t t : sizes) {
        fp8bl_qkv g = base;
        g.eps = e;
        g.tokens = 1 + (t & 3);
        g.q.token_stride = g.k.token_stride = g.v.token_stride = s;
        g.q.head_stride = g.k.head_stride = g.q_out.head_stride = t;
        all(g);
        g.tokens = ((int64_t)1 << 31) - 1;
        g.q_heads = g.k_heads = 4096;
        all(g);
      }
  expect(refused(fp8_qk_norm_rope(nullptr, nullptr)) && refused(fp8_kv_load(nullptr, nullptr)), "null arguments", 0, 0, 0);
  std::printf("%s: %d failures\n", fail ? "FAILED" : "OK", fail);
  return fail ? 1 : 0;
}
