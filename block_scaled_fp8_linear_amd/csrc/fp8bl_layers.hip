// C ABI of the layer operators (declared in include/fp8bl_layers.h): argument
// validation before any HIP call, workspace sizing and layout, and the order
// of the launches. Nothing here touches tensor data.
#include "fp8bl_layers.h"

#include "fp8bl_arrays.h"
#include "fp8bl_internal.h"

namespace {

using namespace fp8bl::checks;
using fp8bl::gate_current_device;
using fp8bl::kWorkspaceAlign;
using fp8bl::round_up;

constexpr int64_t kMaxLayerDim = (int64_t)1 << 20;   // n and k: either can be a product's reduction
                                                     // and is addressed with 32-bit buffer offsets

int check_sizes(int64_t m, int64_t n, int64_t k, int act) {
  if (act < FP8BL_ACT_NONE || act > FP8BL_ACT_GELU_TANH) return FP8BL_INVALID_ARG;
  if (m < 0 || m >= kMaxDim) return FP8BL_INVALID_ARG;
  const int st = check_nk(n, k);
  if (st != FP8BL_OK) return st;
  if (n > kMaxLayerDim || k > kMaxLayerDim) return FP8BL_INVALID_ARG;
  if (m > 0 && (m * k >= kMaxElems || m * n >= kMaxElems)) return FP8BL_INVALID_ARG;
  return FP8BL_OK;
}

bool sizes_ok(int64_t m, int64_t n, int64_t k) {
  return m > 0 && n > 0 && check_sizes(m, n, k, FP8BL_ACT_NONE) == FP8BL_OK;
}

// Rows of the gradients as the input-gradient product reads them.
int64_t padded(int64_t n) { return (n + 7) / 8 * 8; }

// Backward workspace: padded copies of the gradients where n % 8 != 0, the
// column sums' partials, the product's split partials, each 256-byte aligned.
size_t pad_bytes(int64_t m, int64_t n) {
  return n % 8 == 0 ? 0 : round_up((size_t)m * padded(n) * 2, kWorkspaceAlign);
}

template <typename T>
T* at(void* ws, size_t off) { return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off); }

}  // namespace

FP8BL_EXPORT size_t fp8_block_linear_act_workspace_size(int64_t m, int64_t n, int64_t k) {
  return sizes_ok(m, n, k) ? fp8bl::linear_act_bytes(m, n, k) : 0;
}

FP8BL_EXPORT int fp8_block_linear_act(const uint16_t* x, const uint8_t* q, const float* scale_inv,
                                      const uint16_t* bias, const uint16_t* residual, uint16_t* z,
                                      uint16_t* y, int64_t m, int64_t n, int64_t k, int act,
                                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int st = check_sizes(m, n, k, act);
  if (st != FP8BL_OK) return st;
  if (m == 0 || n == 0) return FP8BL_OK;
  const size_t mn = (size_t)m * n * 2;
  const std::initializer_list<Array> arrays = {
      {x, (size_t)m * k * 2, 16, false},
      {q, (size_t)n * k, 16, false},
      {scale_inv, grid_elems(n, k) * 4, 4, false},
      {bias, bias ? (size_t)n * 2 : 0, 16, false},
      {residual, residual ? mn : 0, 16, false, y},
      {z, z ? mn : 0, 16, true},
      {y, mn, 16, true}};
  st = check_arrays(arrays);
  if (st != FP8BL_OK) return st;
  const size_t need = fp8_block_linear_act_workspace_size(m, n, k);
  st = check_workspace(workspace, workspace_bytes, need, arrays);
  if (st != FP8BL_OK) return st;
  st = gate_current_device();
  if (st != FP8BL_OK) return st;
  const fp8bl::LayerEpilogue ep{bias, residual, z, nullptr, nullptr, act};
  return hip_status(
      fp8bl::launch_linear_act(x, q, scale_inv, y, ep, m, n, k, workspace, workspace_bytes, stream));
}

FP8BL_EXPORT size_t fp8_block_linear_act_backward_workspace_size(int64_t m, int64_t n, int64_t k) {
  if (!sizes_ok(m, n, k)) return 0;
  return pad_bytes(m, n) + fp8bl::column_sum_bytes(m, n) + fp8bl::input_gradient_bytes(m, n, k, 1);
}

FP8BL_EXPORT int fp8_block_linear_act_backward(const uint16_t* dy, const uint16_t* z, const uint8_t* q,
                                               const float* scale_inv, uint16_t* dz, float* dbias,
                                               uint16_t* dx, int64_t m, int64_t n, int64_t k, int act,
                                               void* workspace, size_t workspace_bytes,
                                               hipStream_t stream) {
  int st = check_sizes(m, n, k, act);
  if (st != FP8BL_OK) return st;
  const bool has_act = act != FP8BL_ACT_NONE;
  if (!has_act && (z != nullptr || dz != nullptr)) return FP8BL_INVALID_ARG;
  const bool product = m > 0 && n > 0 && dx != nullptr;
  const size_t mn = (size_t)m * n * 2;
  const std::initializer_list<Array> arrays = {
      {dy, mn, 16, false},
      {z, has_act ? mn : 0, 16, false},
      {q, product ? (size_t)n * k : 0, 16, false},
      {scale_inv, product ? grid_elems(n, k) * 4 : 0, 4, false},
      {dz, has_act ? mn : 0, 16, true},
      {dbias, dbias ? (size_t)n * 4 : 0, 4, true},
      {dx, dx ? (size_t)m * k * 2 : 0, 16, true}};
  st = check_arrays(arrays);
  if (st != FP8BL_OK) return st;
  const size_t need = fp8_block_linear_act_backward_workspace_size(m, n, k);
  st = check_workspace(workspace, workspace_bytes, need, arrays);
  if (st != FP8BL_OK) return st;
  if (m == 0 && (dbias == nullptr || n == 0)) return FP8BL_OK;
  if (n == 0 && dx == nullptr) return FP8BL_OK;
  st = gate_current_device();
  if (st != FP8BL_OK) return st;
  // empty sums are zeros
  if (m == 0) return hip_status(fp8bl::launch_fill_zero(dbias, (size_t)n * 4, stream));
  if (n == 0) return hip_status(fp8bl::launch_fill_zero(dx, (size_t)m * k * 2, stream));

  const bool pad = n % 8 != 0;
  uint16_t* const copy = pad && product ? at<uint16_t>(workspace, 0) : nullptr;
  float* const part = at<float>(workspace, pad_bytes(m, n));
  if (has_act || dbias != nullptr || copy != nullptr) {
    const hipError_t e = fp8bl::launch_act_backward(dy, z, dz, copy, padded(n), dbias, part, m, n, act, stream);
    if (e != hipSuccess) return FP8BL_HIP_ERROR;
  }
  if (!product) return FP8BL_OK;
  const size_t off = pad_bytes(m, n) + fp8bl::column_sum_bytes(m, n);
  return hip_status(fp8bl::launch_input_gradient(
      copy ? copy : has_act ? dz : dy, q, scale_inv, nullptr, nullptr, nullptr, padded(n), dx, m, n, k,
      at<void>(workspace, off), need - off, stream));
}

FP8BL_EXPORT size_t fp8_block_glu_workspace_size(int64_t m, int64_t n, int64_t k) {
  return sizes_ok(m, n, k) ? fp8bl::glu_bytes(m, n, k) : 0;
}

FP8BL_EXPORT int fp8_block_glu(const uint16_t* x, const uint8_t* q_gate, const float* scale_inv_gate,
                               const uint8_t* q_up, const float* scale_inv_up, uint16_t* g, uint16_t* u,
                               uint16_t* h, int64_t m, int64_t n, int64_t k, int act, void* workspace,
                               size_t workspace_bytes, hipStream_t stream) {
  int st = check_sizes(m, n, k, act);
  if (st != FP8BL_OK) return st;
  if ((g == nullptr) != (u == nullptr)) return FP8BL_INVALID_ARG;
  if (m == 0 || n == 0) return FP8BL_OK;
  const size_t mn = (size_t)m * n * 2, w = (size_t)n * k, sc = grid_elems(n, k) * 4;
  const std::initializer_list<Array> arrays = {
      {x, (size_t)m * k * 2, 16, false},
      {q_gate, w, 16, false},
      {scale_inv_gate, sc, 4, false},
      {q_up, w, 16, false},
      {scale_inv_up, sc, 4, false},
      {g, g ? mn : 0, 16, true},
      {u, u ? mn : 0, 16, true},
      {h, mn, 16, true}};
  st = check_arrays(arrays);
  if (st != FP8BL_OK) return st;
  const size_t need = fp8_block_glu_workspace_size(m, n, k);
  st = check_workspace(workspace, workspace_bytes, need, arrays);
  if (st != FP8BL_OK) return st;
  st = gate_current_device();
  if (st != FP8BL_OK) return st;
  const fp8bl::LayerEpilogue ep{nullptr, nullptr, nullptr, g, u, act};
  return hip_status(fp8bl::launch_glu(x, q_gate, scale_inv_gate, q_up, scale_inv_up, h, ep, m, n, k,
                                      workspace, workspace_bytes, stream));
}

FP8BL_EXPORT size_t fp8_block_glu_backward_workspace_size(int64_t m, int64_t n, int64_t k) {
  if (!sizes_ok(m, n, k)) return 0;
  return 2 * pad_bytes(m, n) + fp8bl::input_gradient_bytes(m, n, k, 2);
}

FP8BL_EXPORT int fp8_block_glu_backward(const uint16_t* dh, const uint16_t* g, const uint16_t* u,
                                        const uint8_t* q_gate, const float* scale_inv_gate,
                                        const uint8_t* q_up, const float* scale_inv_up, uint16_t* dg,
                                        uint16_t* du, uint16_t* dx, int64_t m, int64_t n, int64_t k,
                                        int act, void* workspace, size_t workspace_bytes,
                                        hipStream_t stream) {
  int st = check_sizes(m, n, k, act);
  if (st != FP8BL_OK) return st;
  const bool product = m > 0 && n > 0 && dx != nullptr;
  const size_t mn = (size_t)m * n * 2;
  const size_t w = product ? (size_t)n * k : 0, sc = product ? grid_elems(n, k) * 4 : 0;
  const std::initializer_list<Array> arrays = {
      {dh, mn, 16, false},
      {g, mn, 16, false},
      {u, mn, 16, false},
      {q_gate, w, 16, false},
      {scale_inv_gate, sc, 4, false},
      {q_up, w, 16, false},
      {scale_inv_up, sc, 4, false},
      {dg, mn, 16, true},
      {du, mn, 16, true},
      {dx, dx ? (size_t)m * k * 2 : 0, 16, true}};
  st = check_arrays(arrays);
  if (st != FP8BL_OK) return st;
  const size_t need = fp8_block_glu_backward_workspace_size(m, n, k);
  st = check_workspace(workspace, workspace_bytes, need, arrays);
  if (st != FP8BL_OK) return st;
  if (m == 0 || (n == 0 && dx == nullptr)) return FP8BL_OK;
  st = gate_current_device();
  if (st != FP8BL_OK) return st;
  if (n == 0) return hip_status(fp8bl::launch_fill_zero(dx, (size_t)m * k * 2, stream));

  const bool pad = n % 8 != 0 && product;
  uint16_t* const cg = pad ? at<uint16_t>(workspace, 0) : nullptr;
  uint16_t* const cu = pad ? at<uint16_t>(workspace, pad_bytes(m, n)) : nullptr;
  const hipError_t e = fp8bl::launch_glu_backward(dh, g, u, dg, du, cg, cu, m, n, act, stream);
  if (e != hipSuccess) return FP8BL_HIP_ERROR;
  if (!product) return FP8BL_OK;
  const size_t off = 2 * pad_bytes(m, n);
  return hip_status(fp8bl::launch_input_gradient(pad ? cg : dg, q_gate, scale_inv_gate, pad ? cu : du,
                                                 q_up, scale_inv_up, padded(n), dx, m, n, k,
                                                 at<void>(workspace, off), need - off, stream));
}
