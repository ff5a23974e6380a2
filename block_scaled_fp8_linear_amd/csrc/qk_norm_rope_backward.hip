// Backward pass of the norm and rotation of query and key heads. For each head,
// with dn the gradient turned by -theta, r = 1 / sqrt(mean(x^2) + eps) and the
// weight w,
//   u = dn w,   dx = r u - x (r^3 mean(u x)),   dw += dn x r.
// Both sums over the head run together, so each head is read and written once.
// A wave takes a token (or a part of its heads) at a time and keeps its share
// of the weights' gradients in registers until its last one; a second kernel
// adds the workgroups' sums in a fixed order. Bound by the heads' bytes: 8192
// tokens of 72 heads of 128 take 88.5 us (5.1 TB/s), of which the second kernel and
// its launch are 4; 77 tokens of 18 heads of 80 take 7.0, the two launches' own
// time.
#include "fp8bl_ops.h"
#include "qkv_device.h"

namespace fp8bl {

namespace {

struct BackArgs {
  HeadView x[2], dy[2], dx[2];     // q, k
  TurnArgs t;
  int parts;
  float* part;                     // [workgroups][2][dim]
};

template <int L, bool INTER, bool PAST>
__device__ __forceinline__ void back_heads(const BackArgs& g, int which, const uint16_t* weight, int token, int first,
                                           int last, int lane, const Chunk& ch, const float (&c)[8],
                                           const float (&s)[8], float (&dw)[8]) {
  const int dim = g.t.dim, col = 8 * (lane % L);
  const bool mine = col < dim;
  float w[8];
  unpack8(mine ? *reinterpret_cast<const u32x4*>(weight + col) : u32x4{0, 0, 0, 0}, w);
  const HeadView &xv = g.x[which], &yv = g.dy[which], &ov = g.dx[which];
  const uint16_t* const xp = xv.p + token * xv.ts + col;
  const uint16_t* const yp = yv.p + token * yv.ts + col;
  uint16_t* const op = ov.p + token * ov.ts + col;
  const float inv_dim = 1.0f / (float)dim;
  // one step's loads of x and of the gradient on their way at a time: with two the
  // same (8192 tokens of 72 heads 98 us through the caches), for more registers
  for (int h0 = first; h0 < last; h0 += 64 / L) {
    const int h = h0 + lane / L;
    const bool live = mine && h < last;
    const u32x4 xr = live ? get8<PAST>(xp + h * xv.hs) : u32x4{0, 0, 0, 0};
    const u32x4 yr = live ? get8<PAST>(yp + h * yv.hs) : u32x4{0, 0, 0, 0};
    float x[8], y[8], o[8], sq = 0.0f, ux = 0.0f;
    unpack8(xr, x);
    unpack8(yr, y);
    unpack8(other_members<INTER>(yr, ch.partner), o);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = __builtin_fmaf(y[i], c[i], -(o[i] * s[i]));        // dn
      sq = __builtin_fmaf(x[i], x[i], sq);
      ux = __builtin_fmaf(y[i] * w[i], x[i], ux);
    }
    float mean = head_sum<L>(sq) * inv_dim + (float)g.t.eps;
    int by = 0;
    if (__builtin_expect(!norm_in_range(mean), 0)) {
      // with x scaled, r and the gradient of x come scaled the other way
      by = norm_exponent<L>(x, g.t.eps);
      ux = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = ldexpf(x[i], -by);
        ux = __builtin_fmaf(y[i] * w[i], x[i], ux);
      }
      mean = norm_scaled<L>(x, inv_dim, g.t.eps, by);
    }
    const float r = rsqrtf(mean);
    const float along = head_sum<L>(ux) * inv_dim * r * r;
    // a head that is not there leaves zeros in the sums, whatever r is
    const float rl = live ? r : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[i] = __builtin_fmaf(y[i] * rl, x[i], dw[i]);
      o[i] = r * __builtin_fmaf(-x[i], along, y[i] * w[i]);
    }
    if (__builtin_expect(by != 0, 0)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = ldexpf(o[i], -by);
    }
    if (live) put8<PAST>(op + h * ov.hs, pack8(o));
  }
}

template <int L, bool INTER, bool PAST>
__global__ __launch_bounds__(kQkvThreads)
void back_kernel(BackArgs g) {
  __shared__ float2 tables[kQkvWaves][FP8BL_MAX_PAIRS];
  __shared__ float sums[kQkvWaves][2][8 * L];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Chunk ch = chunk_of<INTER>(lane, lane % L, g.t.pairs);
  float dwq[8] = {}, dwk[8] = {};
  constexpr int G = 64 / L;
  const int sq = (g.x[0].heads + G - 1) / G, sk = (g.x[1].heads + G - 1) / G;
  const int units = g.t.tokens * g.parts;
  for (int64_t u = (int64_t)blockIdx.x * kQkvWaves + wave; u < units; u += (int64_t)gridDim.x * kQkvWaves) {
    const int token = (int)u / g.parts, part = (int)u % g.parts;
    wave_sync();
    for (int p = lane; p < g.t.pairs; p += 64) tables[wave][p] = turn_of(g.t, g.t.axis[p], p, token);
    wave_sync();
    float c[8], s[8];
    turn_factors<INTER>(tables[wave], ch, c, s);
    const int s0 = (sq + sk) * part / g.parts, s1 = (sq + sk) * (part + 1) / g.parts;
    if (s0 < sq)
      back_heads<L, INTER, PAST>(g, 0, g.t.wq, token, s0 * G, min(min(s1, sq) * G, g.x[0].heads), lane, ch, c, s, dwq);
    if (s1 > sq)
      back_heads<L, INTER, PAST>(g, 1, g.t.wk, token, max(s0 - sq, 0) * G, min((s1 - sq) * G, g.x[1].heads), lane, ch,
                                 c, s, dwk);
  }
  // over the heads a wave holds side by side, then over the waves
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int off = L; off < 64; off *= 2) {
      dwq[i] += __shfl_xor(dwq[i], off, 64);
      dwk[i] += __shfl_xor(dwk[i], off, 64);
    }
    if (lane < L) {
      sums[wave][0][8 * lane + i] = dwq[i];
      sums[wave][1][8 * lane + i] = dwk[i];
    }
  }
  __syncthreads();
  for (int e = tid; e < 2 * g.t.dim; e += kQkvThreads) {
    const int which = e >= g.t.dim, col = e - which * g.t.dim;
    float t = sums[0][which][col];
#pragma unroll
    for (int w = 1; w < kQkvWaves; ++w) t += sums[w][which][col];
    g.part[(size_t)blockIdx.x * 2 * g.t.dim + e] = t;
  }
}

// Sum over the workgroups: 16 columns a workgroup, 64 rows of the partials at
// a time, kRows loads of a thread on their way.
__global__ __launch_bounds__(1024)
void back_sum_kernel(const float* __restrict__ part, int blocks, int dim, float* dwq, float* dwk) {
  __shared__ float sums[64][17];
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4, e = blockIdx.x * 16 + col;
  constexpr int kRows = 8;
  float t = 0.0f;
  for (int b0 = row; b0 < blocks; b0 += 64 * kRows) {
    float v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int b = b0 + 64 * i;
      v[i] = b < blocks && e < 2 * dim ? part[(size_t)b * 2 * dim + e] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) t += v[i];
  }
  sums[row][col] = t;
  __syncthreads();
  for (int half = 32; half >= 1; half /= 2) {
    if (row < half) sums[row][col] += sums[row + half][col];
    __syncthreads();
  }
  if (row == 0 && e < 2 * dim) {
    float* const out = e < dim ? dwq : dwk;
    if (out != nullptr) out[e < dim ? e : e - dim] = sums[0][col];
  }
}

// Workgroups: fixed by the sizes alone, for results that are the same on every
// device and call. Four a compute unit; with 512, 1024 and 2048 of them 8192 tokens of
// 72 heads of 128 take 99, 87 and 91 us, of 18 heads of 80 30.1, 24.0 and 27.0, of
// three heads of 64 16.6, 15.1 and 18.9; 512 tokens of 72 heads 12.5, 14.0 and 20.3, 2048
// of 18 heads of 80 12.4, 13.0 and 18.1.
constexpr int64_t kBackBlocks = 1024;

int back_parts(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim) {
  const int64_t g = 64 / head_lanes(dim), steps = (q_heads + g - 1) / g + (k_heads + g - 1) / g;
  int64_t parts = 4 * kBackBlocks / tokens;
  if (parts > steps) parts = steps;
  return parts < 1 ? 1 : (int)parts;
}

int64_t back_blocks(int64_t tokens, int parts) {
  const int64_t blocks = (tokens * parts + kQkvWaves - 1) / kQkvWaves;
  return blocks < kBackBlocks ? blocks : kBackBlocks;
}

struct Back {
  const fp8bl_qkv& a;
  float* part;
  hipStream_t stream;
  template <int L, bool INTER>
  hipError_t launch() {
    BackArgs g{{head_view(a.q, a.q_heads), head_view(a.k, a.k_heads)},
               {head_view(a.dq, a.q_heads), head_view(a.dk, a.k_heads)},
               {head_view(a.q_out, a.q_heads), head_view(a.k_out, a.k_heads)},
               turn_args(a),
               back_parts(a.tokens, a.q_heads, a.k_heads, a.head_dim),
               part};
    const int blocks = (int)back_blocks(a.tokens, g.parts);
    if (past_caches(a.tokens * (a.q_heads + a.k_heads) * a.head_dim * 6))
      hipLaunchKernelGGL((back_kernel<L, INTER, true>), dim3(blocks), dim3(kQkvThreads), 0, stream, g);
    else
      hipLaunchKernelGGL((back_kernel<L, INTER, false>), dim3(blocks), dim3(kQkvThreads), 0, stream, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || (a.dq_weight == nullptr && a.dk_weight == nullptr)) return e;
    hipLaunchKernelGGL(back_sum_kernel, dim3((uint32_t)((2 * a.head_dim + 15) / 16)), dim3(1024), 0, stream, part,
                       blocks, (int)a.head_dim, a.dq_weight, a.dk_weight);
    return hipGetLastError();
  }
  template <int L>
  hipError_t run() {
    return a.interleaved ? launch<L, true>() : launch<L, false>();
  }
};

}  // namespace

size_t qk_backward_bytes(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim) {
  const int64_t blocks = back_blocks(tokens, back_parts(tokens, q_heads, k_heads, head_dim));
  return round_up((size_t)blocks * 2 * head_dim * sizeof(float), kWorkspaceAlign);
}

hipError_t launch_qk_norm_rope_backward(const fp8bl_qkv& a, float* part, hipStream_t stream) {
  return with_lanes(a.head_dim, Back{a, part, stream});
}

}  // namespace fp8bl
