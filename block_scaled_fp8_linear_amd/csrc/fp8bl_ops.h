// Internal launchers behind fp8bl_int8.h and fp8bl_qkv.h. Every launcher
// assumes its arguments were validated by the ABI layer.
#pragma once

#include "fp8bl_internal.h"
#include "int8_plan.h"

struct fp8bl_qkv;

namespace fp8bl {

// ---- 8-bit integer linear.
hipError_t launch_int8_quantize(const float* x, int8_t* q, float* scale, int64_t m, int64_t k, hipStream_t stream);
hipError_t launch_int8_quantize(const uint16_t* x, int8_t* q, float* scale, int64_t m, int64_t k,
                                hipStream_t stream);
size_t int8_gemm_bytes(int64_t m, int64_t n, int64_t k);
hipError_t launch_int8_gemm(const int8_t* xq, const float* xs, const int8_t* wq, const float* ws,
                            const uint16_t* bias, uint16_t* y, int64_t m, int64_t n, int64_t k, void* workspace,
                            hipStream_t stream);
// At up to kInt8SkinnyRows rows; and from one row of bf16, quantized on the way
// where int8_skinny_quantizes says so.
size_t int8_skinny_bytes(int64_t m, int64_t n, int64_t k);
hipError_t launch_int8_skinny(const int8_t* xq, const float* xs, const int8_t* wq, const float* ws,
                              const uint16_t* bias, uint16_t* y, int64_t m, int64_t n, int64_t k, void* workspace,
                              hipStream_t stream);
hipError_t launch_int8_skinny_bf16(const uint16_t* x, const int8_t* wq, const float* ws, const uint16_t* bias,
                                   uint16_t* y, int64_t n, int64_t k, hipStream_t stream);
// Sum of K splits' partials (slabs of partial_slab(m, n)) with the epilogue.
hipError_t launch_int8_join(const int32_t* part, const float* xs, const float* ws, const uint16_t* bias, uint16_t* y,
                            int splits, int64_t m, int64_t n, hipStream_t stream);

// ---- From the QKV projection to its cache.
hipError_t launch_qk_norm_rope(const fp8bl_qkv& a, hipStream_t stream);
size_t qk_backward_bytes(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim);
hipError_t launch_qk_norm_rope_backward(const fp8bl_qkv& a, float* part, hipStream_t stream);
hipError_t launch_kv_store(const fp8bl_qkv& a, hipStream_t stream);
hipError_t launch_kv_load(const fp8bl_qkv& a, hipStream_t stream);
hipError_t launch_qk_norm_rope_store(const fp8bl_qkv& a, hipStream_t stream);

}  // namespace fp8bl
