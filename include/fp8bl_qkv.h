/*
 * fp8bl_qkv.h — from a block's QKV projection to its cache: the norm and the
 * position rotation of each query and key head, and a cache of keys and values
 * in E4M3 with one scale for each token and head.
 *
 * What fp8bl.h says of its calls holds here: device pointers owned by the
 * caller, bf16 as 16-bit patterns, work enqueued on `stream`, no allocation
 * and no synchronisation, every argument error reported by the return code
 * before anything is launched. What differs:
 *   - a call's arguments come in one structure, of which each call reads the
 *     members that it names and no others;
 *   - q, k, v and their like are views of a larger array as well as arrays of
 *     their own: [tokens, heads, head_dim] with the last axis contiguous and a
 *     stride for each of the others, in elements, multiples of 8, not negative
 *     and at most 2^40. 16-byte aligned. An output's elements are all distinct (its
 *     heads lie inside its token stride or its tokens inside its head stride)
 *     and overlap no other array. Two arrays with the same token stride whose
 *     tokens lie beside each other, as q, k and v in one projection's output,
 *     do not overlap;
 *   - head_dim is a multiple of 8 from 16 to 256; tokens, heads and cache rows
 *     are below 2^31, heads at most 4096.
 */
#ifndef FP8BL_QKV_H
#define FP8BL_QKV_H

#include "fp8bl.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FP8BL_MAX_AXES 8
#define FP8BL_MAX_PAIRS 128

/* bf16 [tokens, heads, head_dim]. */
typedef struct fp8bl_heads {
  uint16_t* data;
  int64_t token_stride;
  int64_t head_stride;
} fp8bl_heads;

typedef struct fp8bl_qkv {
  int64_t tokens;
  int64_t q_heads;
  int64_t k_heads;             /* v's too */
  int64_t head_dim;
  fp8bl_heads q, k, v;         /* as the projection wrote them */
  fp8bl_heads q_out, k_out, v_out;
  fp8bl_heads dq, dk;          /* gradients of what fp8_qk_norm_rope wrote */
  /* norm and rotation */
  const uint16_t* q_weight;    /* [head_dim] bf16 */
  const uint16_t* k_weight;    /* [head_dim] bf16 */
  float* dq_weight;            /* [head_dim] fp32 */
  float* dk_weight;            /* [head_dim] fp32 */
  const int32_t* positions;    /* [axes, tokens] */
  const float* inv_freq;       /* [pairs] fp32 */
  int64_t axes;                /* 1 .. FP8BL_MAX_AXES */
  int64_t pairs;               /* 1 .. head_dim / 2 */
  int64_t interleaved;         /* 0 or 1 */
  double eps;                  /* >= 0 */
  /* cache */
  const int32_t* slots;        /* [tokens]: the cache row of each token */
  uint8_t* k_cache;            /* [cache_rows, k_heads, head_dim] E4M3 */
  uint8_t* v_cache;
  float* k_scale;              /* [cache_rows, k_heads] fp32 */
  float* v_scale;
  int64_t cache_rows;
  uint8_t axis[FP8BL_MAX_PAIRS]; /* axis[i] < axes: the axis that pair i turns by */
} fp8bl_qkv;

/* Norm and rotation of each head x of q and k:
 *   n = x / sqrt(mean(x^2) + eps) * weight
 *   theta_i = positions[axis[i], token] * inv_freq[i]
 *   pair i (a, b) of n -> (a cos theta_i - b sin theta_i, b cos theta_i + a sin theta_i)
 * Pair i is elements i and i + pairs, or 2 i and 2 i + 1 where `interleaved`;
 * elements from 2 * pairs on are not turned. `pairs` is a multiple of 8, or of
 * 4 where `interleaved`. theta is the exact product, reduced in fp64 (to 2^-53
 * below 2^40 radians); all else is fp32, and the result is rounded to bf16 once.
 * A head whose mean(x^2) + eps lies outside 2^-32 .. 2^64 is scaled by a power
 * of two first, so that any finite head and any eps give what the formula says; a
 * head of zeros with an eps of 0 gives zeros. A head with a value that is not
 * finite gives unspecified values of its own.
 * Reads tokens, q_heads, k_heads, head_dim, q, k, q_weight, k_weight,
 * positions, inv_freq, axes, pairs, interleaved, eps, axis; writes q_out (which
 * may be q) and k_out (which may be k). inv_freq and positions 4-byte, weights
 * 16-byte aligned. */
int fp8_qk_norm_rope(const fp8bl_qkv* args, hipStream_t stream);

/* Its backward pass. With dn the turn of dq (dk) by -theta, r = 1 / sqrt(mean(x^2) + eps),
 * u = dn * weight:
 *   gradient of x       r (u - x r^2 mean(u x))          -> q_out, k_out
 *   gradient of weight  sum over tokens and heads of dn x r  -> dq_weight, dk_weight
 * Reads what fp8_qk_norm_rope reads, and dq and dk; writes q_out (which may be
 * dq), k_out (which may be dk), and dq_weight and dk_weight (4-byte aligned),
 * each of which may be NULL. A head of zeros with an eps of 0 gives zeros here
 * too, and adds nothing to the weight's gradient. Sums in fp32 in an order fixed
 * by the sizes: the same bits on every call. The workspace (256-byte aligned, of
 * at least the queried size) needs no initialisation; calls that share one must
 * be ordered. */
size_t fp8_qk_norm_rope_backward_workspace_size(int64_t tokens, int64_t q_heads, int64_t k_heads,
                                                int64_t head_dim);
int fp8_qk_norm_rope_backward(const fp8bl_qkv* args, void* workspace, size_t workspace_bytes,
                              hipStream_t stream);

/* Keys and values into the cache, for each token and head
 *   S = fl32(max |x| / 448)  (1.0 where that is 0),
 *   code = nearest finite E4M3 to fl32(x / S), ties to even, saturating,
 * as fp8_act_quantize does for its groups. Row slots[i] of the cache receives
 * token i; a token whose slot is negative or not below cache_rows is padding
 * and is not stored. Where tokens of a call have the same slot, the last of
 * them is stored. Other rows of the cache are left as they were. At most
 * 65536 tokens. Non-finite values give unspecified codes in their own head.
 * Reads tokens, k_heads, head_dim, k, v, slots, cache_rows; writes k_cache and
 * v_cache (16-byte aligned), k_scale and v_scale (4-byte aligned). */
int fp8_kv_store(const fp8bl_qkv* args, hipStream_t stream);

/* Rows of the cache back as bf16_rne(fl32(e4m3(code) * S)); a token whose
 * slot is outside the cache reads as zeros. The same slot may be read by many
 * tokens. Reads tokens, k_heads, head_dim, slots, k_cache, v_cache, k_scale,
 * v_scale, cache_rows; writes k_out and v_out. */
int fp8_kv_load(const fp8bl_qkv* args, hipStream_t stream);

/* fp8_qk_norm_rope and fp8_kv_store in one pass: q_out as there, and the cache
 * receives v and the normed and turned k, which is computed in fp64 and quantized
 * from there, S = fl32(max |k| / 448) and the code nearest to fl32(k / S) (storing
 * a k_out rounds it to bf16 first). Reads and writes what the two do, but for
 * k_out. At most 65536 tokens. */
int fp8_qk_norm_rope_store(const fp8bl_qkv* args, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BL_QKV_H */
