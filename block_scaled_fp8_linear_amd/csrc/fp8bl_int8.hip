// C ABI of the 8-bit integer linear (declared in include/fp8bl_int8.h):
// argument validation before any HIP call, workspace layout, and the order of
// the launches. Nothing here touches tensor data.
#include "fp8bl_int8.h"

#include "fp8bl_arrays.h"
#include "fp8bl_ops.h"

namespace {

using namespace fp8bl::checks;
using fp8bl::gate_current_device;
using fp8bl::kWorkspaceAlign;
using fp8bl::round_up;

constexpr int64_t kMaxN = (int64_t)1 << 20;         // rows of a tile are addressed with 32-bit buffer offsets
constexpr int64_t kMaxK = ((int64_t)1 << 17) - 16;  // (2^17 - 1) 2^14 < 2^31: a sum of products of -128 fits

int check_rows(int64_t m, int64_t k) {
  if (m < 0 || m >= kMaxDim || k <= 0 || k % 16 != 0 || k > kMaxK) return FP8BL_INVALID_ARG;
  return m * k >= kMaxElems ? FP8BL_INVALID_ARG : FP8BL_OK;
}

int check_sizes(int64_t m, int64_t n, int64_t k) {
  const int st = check_rows(m, k);
  if (st != FP8BL_OK) return st;
  if (n < 0 || n > kMaxN || n * k >= kMaxElems || m * n >= kMaxElems) return FP8BL_INVALID_ARG;
  return FP8BL_OK;
}

bool sizes_ok(int64_t m, int64_t n, int64_t k) { return m > 0 && n > 0 && check_sizes(m, n, k) == FP8BL_OK; }

// Workspace of int8_linear_bf16: the codes and the scales of x, then what the
// product needs, each 256-byte aligned.
size_t codes_bytes(int64_t m, int64_t k) { return round_up((size_t)m * k, kWorkspaceAlign); }
size_t scales_bytes(int64_t m) { return round_up((size_t)m * 4, kWorkspaceAlign); }

template <typename T>
int quantize(const T* x, int8_t* q, float* scale, int64_t m, int64_t k, hipStream_t stream) {
  int st = check_rows(m, k);
  if (st != FP8BL_OK) return st;
  if (m == 0) return FP8BL_OK;
  st = check_arrays({{x, (size_t)m * k * sizeof(T), 16, false},
                     {q, (size_t)m * k, 16, true},
                     {scale, (size_t)m * 4, 4, true}});
  if (st != FP8BL_OK) return st;
  st = gate_current_device();
  if (st != FP8BL_OK) return st;
  return hip_status(fp8bl::launch_int8_quantize(x, q, scale, m, k, stream));
}

}  // namespace

FP8BL_EXPORT int int8_row_quantize(const float* x, int8_t* q, float* scale, int64_t m, int64_t k,
                                   hipStream_t stream) {
  return quantize(x, q, scale, m, k, stream);
}

FP8BL_EXPORT int int8_row_quantize_bf16(const uint16_t* x, int8_t* q, float* scale, int64_t m, int64_t k,
                                        hipStream_t stream) {
  return quantize(x, q, scale, m, k, stream);
}

FP8BL_EXPORT size_t int8_linear_workspace_size(int64_t m, int64_t n, int64_t k) {
  return sizes_ok(m, n, k) ? fp8bl::int8_gemm_bytes(m, n, k) : 0;
}

FP8BL_EXPORT int int8_linear(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                             const uint16_t* bias, uint16_t* y, int64_t m, int64_t n, int64_t k,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int st = check_sizes(m, n, k);
  if (st != FP8BL_OK) return st;
  if (m == 0 || n == 0) return FP8BL_OK;
  const std::initializer_list<Array> arrays = {{xq, (size_t)m * k, 16, false},
                                               {x_scale, (size_t)m * 4, 4, false},
                                               {wq, (size_t)n * k, 16, false},
                                               {w_scale, (size_t)n * 4, 4, false},
                                               {bias, bias ? (size_t)n * 2 : 0, 16, false},
                                               {y, (size_t)m * n * 2, 16, true}};
  st = check_arrays(arrays);
  if (st != FP8BL_OK) return st;
  st = check_workspace(workspace, workspace_bytes, fp8bl::int8_gemm_bytes(m, n, k), arrays);
  if (st != FP8BL_OK) return st;
  st = gate_current_device();
  if (st != FP8BL_OK) return st;
  return hip_status(fp8bl::launch_int8_gemm(xq, x_scale, wq, w_scale, bias, y, m, n, k, workspace, stream));
}

FP8BL_EXPORT size_t int8_linear_bf16_workspace_size(int64_t m, int64_t n, int64_t k) {
  if (!sizes_ok(m, n, k)) return 0;
  return codes_bytes(m, k) + scales_bytes(m) + fp8bl::int8_gemm_bytes(m, n, k);
}

FP8BL_EXPORT int int8_linear_bf16(const uint16_t* x, const int8_t* wq, const float* w_scale,
                                  const uint16_t* bias, uint16_t* y, int64_t m, int64_t n, int64_t k,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int st = check_sizes(m, n, k);
  if (st != FP8BL_OK) return st;
  if (m == 0 || n == 0) return FP8BL_OK;
  const std::initializer_list<Array> arrays = {{x, (size_t)m * k * 2, 16, false},
                                               {wq, (size_t)n * k, 16, false},
                                               {w_scale, (size_t)n * 4, 4, false},
                                               {bias, bias ? (size_t)n * 2 : 0, 16, false},
                                               {y, (size_t)m * n * 2, 16, true}};
  st = check_arrays(arrays);
  if (st != FP8BL_OK) return st;
  st = check_workspace(workspace, workspace_bytes, int8_linear_bf16_workspace_size(m, n, k), arrays);
  if (st != FP8BL_OK) return st;
  st = gate_current_device();
  if (st != FP8BL_OK) return st;
  if (fp8bl::int8_skinny_quantizes(m, k))
    return hip_status(fp8bl::launch_int8_skinny_bf16(x, wq, w_scale, bias, y, n, k, stream));
  uint8_t* const w = static_cast<uint8_t*>(workspace);
  int8_t* const xq = reinterpret_cast<int8_t*>(w);
  float* const xs = reinterpret_cast<float*>(w + codes_bytes(m, k));
  const hipError_t e = fp8bl::launch_int8_quantize(x, xq, xs, m, k, stream);
  if (e != hipSuccess) return FP8BL_HIP_ERROR;
  return hip_status(fp8bl::launch_int8_gemm(xq, xs, wq, w_scale, bias, y, m, n, k,
                                            w + codes_bytes(m, k) + scales_bytes(m), stream));
}
