/*
 * fp8bl_layers.h — layer operators of the block-scaled FP8 linear library:
 * the linear and the gated pair with the epilogues a transformer block puts
 * on them, and the backward pass of both through the frozen weight.
 *
 * Everything fp8bl.h says of its calls holds here: device pointers owned by
 * the caller, bf16 as 16-bit patterns, row-major contiguous arrays, work
 * enqueued on `stream`, no allocation and no synchronisation, every argument
 * error reported by the return code before anything is launched. Pointers are
 * 16-byte aligned (scale grids 4-byte, workspaces 256-byte). What differs:
 *   - n and k are at most 2^20 each (k a positive multiple of 16 as there);
 *   - an empty m or n is not always an empty result: with n == 0 the sums
 *     over n are zero, with m == 0 the sums over rows are zero, and those
 *     outputs are written;
 *   - `workspace` needs no initialisation and is not preserved. Calls that
 *     share one must be ordered (two captured graphs that share one must not
 *     replay at once); it may be NULL when its queried size is 0.
 *
 * W^ is the dequantized weight of fp8_block_dequant. It is a constant of the
 * checkpoint: no call forms a gradient of it. Sums over k, n and rows are
 * held in fp32 in an order fixed by the shape: results are the same bits on
 * every call.
 */
#ifndef FP8BL_LAYERS_H
#define FP8BL_LAYERS_H

#include "fp8bl.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations and their derivatives, evaluated in fp32 (z finite):
 *   NONE       t                                1
 *   RELU       max(t, 0)                        1 for t > 0, else 0
 *   SILU       t p,  p = 1 / (1 + e^-t)         p (1 + t (1 - p))
 *   GELU       t Phi(t)                         Phi(t) + t e^(-t^2/2) / sqrt(2 pi)
 *   GELU_TANH  t p,  p = 1 / (1 + e^-v),        p + t p (1 - p) v',
 *              v = 2 sqrt(2/pi) (t + 0.044715 t^3)   v' = dv/dt  */
enum fp8bl_act {
  FP8BL_ACT_NONE = 0,
  FP8BL_ACT_RELU = 1,
  FP8BL_ACT_SILU = 2,
  FP8BL_ACT_GELU = 3,
  FP8BL_ACT_GELU_TANH = 4
};

/* Linear with bias, activation and residual:
 *   z = x W^T + bias,   y = act(z) + residual,
 * z and y each rounded to bf16 once, from the fp32 sum.
 *   x          [m,k] bf16 (in)
 *   q, scale_inv            the weight [n,k], as for fp8_block_linear (in)
 *   bias       [n] bf16 (in) or NULL
 *   residual   [m,n] bf16 (in) or NULL; may be y itself (added in place),
 *              otherwise it must not overlap an output
 *   z          [m,n] bf16 (out) or NULL: what the backward pass needs
 *   y          [m,n] bf16 (out)
 *   workspace  at least fp8_block_linear_act_workspace_size bytes */
size_t fp8_block_linear_act_workspace_size(int64_t m, int64_t n, int64_t k);
int fp8_block_linear_act(const uint16_t* x, const uint8_t* q, const float* scale_inv,
                         const uint16_t* bias, const uint16_t* residual, uint16_t* z, uint16_t* y,
                         int64_t m, int64_t n, int64_t k, int act, void* workspace,
                         size_t workspace_bytes, hipStream_t stream);

/* Backward pass of fp8_block_linear_act:
 *   dz = dy act'(z),   dbias = sum over rows of dz,   dx = dz W^
 * (the gradient of residual is dy). dbias sums the fp32 dz; dz is rounded to
 * bf16 for the product, which needs bf16 operands, and is the one returned.
 *   dy         [m,n] bf16 (in)
 *   z          [m,n] bf16 (in), as saved; NULL when act is NONE
 *   dz         [m,n] bf16 (out); NULL when act is NONE (dz is dy then)
 *   dbias      [n] fp32 (out, 4-byte aligned) or NULL
 *   dx         [m,k] bf16 (out) or NULL
 *   workspace  at least fp8_block_linear_act_backward_workspace_size bytes */
size_t fp8_block_linear_act_backward_workspace_size(int64_t m, int64_t n, int64_t k);
int fp8_block_linear_act_backward(const uint16_t* dy, const uint16_t* z, const uint8_t* q,
                                  const float* scale_inv, uint16_t* dz, float* dbias, uint16_t* dx,
                                  int64_t m, int64_t n, int64_t k, int act, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream);

/* Gated feed-forward pair:
 *   g = x Wg^T,   u = x Wu^T,   h = act(g) u,
 * each rounded to bf16 once, from the fp32 sums (fp8_block_mlp_gate_up rounds
 * g, u and silu(g) to bf16 on the way, as eager bf16 layers do; h here is
 * nearer the formula and can differ from it in the last bits).
 *   x                   [m,k] bf16 (in)
 *   q_gate, q_up        [n,k] E4M3 (in), scale_inv_* their grids
 *   g, u                [m,n] bf16 (out), both or neither (NULL): what the
 *                       backward pass needs
 *   h                   [m,n] bf16 (out)
 *   workspace           at least fp8_block_glu_workspace_size bytes */
size_t fp8_block_glu_workspace_size(int64_t m, int64_t n, int64_t k);
int fp8_block_glu(const uint16_t* x, const uint8_t* q_gate, const float* scale_inv_gate,
                  const uint8_t* q_up, const float* scale_inv_up, uint16_t* g, uint16_t* u,
                  uint16_t* h, int64_t m, int64_t n, int64_t k, int act, void* workspace,
                  size_t workspace_bytes, hipStream_t stream);

/* Backward pass of fp8_block_glu:
 *   dg = dh u act'(g),   du = dh act(g),   dx = dg Wg^ + du Wu^
 * dg and du are rounded to bf16 once; the products read them so.
 *   dh, g, u            [m,n] bf16 (in), g and u as saved
 *   dg, du              [m,n] bf16 (out)
 *   dx                  [m,k] bf16 (out) or NULL
 *   workspace           at least fp8_block_glu_backward_workspace_size bytes */
size_t fp8_block_glu_backward_workspace_size(int64_t m, int64_t n, int64_t k);
int fp8_block_glu_backward(const uint16_t* dh, const uint16_t* g, const uint16_t* u,
                           const uint8_t* q_gate, const float* scale_inv_gate, const uint8_t* q_up,
                           const float* scale_inv_up, uint16_t* dg, uint16_t* du, uint16_t* dx,
                           int64_t m, int64_t n, int64_t k, int act, void* workspace,
                           size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BL_LAYERS_H */
