/*
 * fp8bl_int8.h — the 8-bit integer linear of the block-scaled FP8 linear
 * library: codes with one fp32 scale for each row (an activation's token, a
 * weight's output channel), multiplied on the integer matrix cores with exact
 * 32-bit sums.
 *
 * Everything fp8bl.h says of its calls holds here: device pointers owned by
 * the caller, bf16 as 16-bit patterns, row-major contiguous arrays, work
 * enqueued on `stream`, no allocation and no synchronisation, every argument
 * error reported by the return code before anything is launched. Pointers are
 * 16-byte aligned (scales 4-byte, workspaces 256-byte). What differs:
 *   - n is at most 2^20, and k (a positive multiple of 16) at most 131056:
 *     there the sum of k products of codes still fits 32 bits, for any codes
 *     (also -128, which the quantizer never writes);
 *   - `workspace` needs no initialisation and is not preserved. Calls that
 *     share one must be ordered (two captured graphs that share one must not
 *     replay at once); it may be NULL when its queried size is 0.
 */
#ifndef FP8BL_INT8_H
#define FP8BL_INT8_H

#include "fp8bl.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Quantization of each row, for the tokens of an activation or the output
 * channels of a weight:
 *   S = fl32(max |x| / 127)  (IEEE division; 1.0 where that is 0),
 *   Q = the integer nearest to fl32(x / S), ties to even, within +-127.
 *   x       [m,k] finite (in)
 *   q       [m,k] int8 (out)
 *   scale   [m] fp32 (out)
 * Bit-exact. A row with a non-finite x gives unspecified codes and scale; the
 * other rows are not touched by it. */
int int8_row_quantize(const float* x, int8_t* q, float* scale, int64_t m, int64_t k,
                      hipStream_t stream);
int int8_row_quantize_bf16(const uint16_t* x, int8_t* q, float* scale, int64_t m, int64_t k,
                           hipStream_t stream);

/* The linear on codes:
 *   y[m,n] = bf16_rne( (sum_k xq[m,k] * wq[n,k]) * (x_scale[m] * w_scale[n]) + bias[n] )
 * The sum is exact in 32 bits whatever its order, so results are the same bits
 * on every call; its conversion, the product of the scales, the product of the
 * two and the sum with the bias are one fp32 rounding each.
 *   xq, x_scale  [m,k] int8 and [m] fp32 (in)
 *   wq, w_scale  [n,k] int8 and [n] fp32 (in)
 *   bias         [n] bf16 (in) or NULL
 *   y            [m,n] bf16 (out, may not overlap)
 *   workspace    at least int8_linear_workspace_size bytes */
size_t int8_linear_workspace_size(int64_t m, int64_t n, int64_t k);
int int8_linear(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                const uint16_t* bias, uint16_t* y, int64_t m, int64_t n, int64_t k, void* workspace,
                size_t workspace_bytes, hipStream_t stream);

/* The whole route from a bf16 activation: int8_row_quantize_bf16, then
 * int8_linear. Same bits as those two calls.
 *   x            [m,k] bf16, finite (in)
 *   workspace    at least int8_linear_bf16_workspace_size bytes (the codes
 *                and scales of x among them) */
size_t int8_linear_bf16_workspace_size(int64_t m, int64_t n, int64_t k);
int int8_linear_bf16(const uint16_t* x, const int8_t* wq, const float* w_scale, const uint16_t* bias,
                     uint16_t* y, int64_t m, int64_t n, int64_t k, void* workspace,
                     size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BL_INT8_H */
