// Elementwise part of the layer operators' backward passes, bound by HBM.
//
//   linear: dz = dy act'(z), dbias[c] = sum over rows of dz[r, c]
//   gated:  dg = dh u act'(g), du = dh act(g)
//
// The products that follow read the gradients in rows of whole 16-byte
// chunks. Where N is no multiple of 8 the kernels also write a copy with
// padded rows (`ld` elements, the padding zero).
#include "fp8bl_act.h"
#include "fp8bl_device.h"
#include "fp8bl_internal.h"

namespace fp8bl {

namespace {

constexpr int kThreads = 256;
constexpr int kColThreads = 32;                      // threads side by side along a row
constexpr int kRowLanes = kThreads / kColThreads;    // rows in hand at once

template <int VEC>
struct Vec;
template <>
struct Vec<8> {
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const u32x4*>(p); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = v[i >> 1];
    return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  __device__ __forceinline__ static void store(uint16_t* p, const float (&f)[8]) {
    const u32x4 o = {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                     pack_bf16x2(f[6], f[7])};
    *reinterpret_cast<u32x4*>(p) = o;
  }
};
template <>
struct Vec<1> {
  uint16_t v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *p; }
  __device__ __forceinline__ float get(int) const { return __uint_as_float((uint32_t)v << 16); }
  __device__ __forceinline__ static void store(uint16_t* p, const float (&f)[1]) {
    *p = __builtin_bit_cast(uint16_t, (__bf16)f[0]);
  }
};

// A workgroup covers 32 * VEC columns and one chunk of rows: thread (rl, cl)
// takes rows rl, rl + 8, ... of the chunk. The column sums of the eight row
// lanes meet in LDS and are added in lane order; the chunks' sums go to
// `part` [chunks, N] and are added in order by the second kernel (no atomics:
// the same bits on every call). dz may be null (act none: dz is dy), the
// padded copy too.
template <int ACT, int VEC>
__global__ __launch_bounds__(kThreads)
void act_backward_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ z,
                         uint16_t* __restrict__ dz, uint16_t* __restrict__ pad, int64_t ld,
                         float* __restrict__ sums, int64_t M, int64_t N, int64_t rows_per_chunk,
                         int col_blocks) {
  __shared__ float red[kRowLanes][kColThreads * VEC + 1];
  const int cl = threadIdx.x % kColThreads, rl = threadIdx.x / kColThreads;
  const int64_t chunk = blockIdx.x / (uint32_t)col_blocks;
  const int64_t col = ((int64_t)(blockIdx.x % (uint32_t)col_blocks) * kColThreads + cl) * VEC;
  const int64_t r1 = min((chunk + 1) * rows_per_chunk, M);
  float sum[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
  if (col < N) {
#pragma unroll 4
    for (int64_t r = chunk * rows_per_chunk + rl; r < r1; r += kRowLanes) {
      Vec<VEC> a, b;
      a.load(dy + r * N + col);
      if constexpr (ACT != kActNone) b.load(z + r * N + col);
      float d[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        d[i] = a.get(i);
        if constexpr (ACT != kActNone) d[i] *= act_grad_f32<ACT>(b.get(i));
        sum[i] += d[i];
      }
      if (ACT != kActNone && dz) Vec<VEC>::store(dz + r * N + col, d);
      if (VEC == 1 && pad) Vec<VEC>::store(pad + r * ld + col, d);
    }
  }
  // the padding of the chunk's rows, by the workgroup that has the last columns
  if (VEC == 1 && pad && col >= N && col < ld)
    for (int64_t r = chunk * rows_per_chunk + rl; r < r1; r += kRowLanes) pad[r * ld + col] = 0;
  if (!sums) return;
#pragma unroll
  for (int i = 0; i < VEC; ++i) red[rl][cl * VEC + i] = sum[i];
  __syncthreads();
  const int64_t c0 = (int64_t)(blockIdx.x % (uint32_t)col_blocks) * kColThreads * VEC;
  for (int c = threadIdx.x; c < kColThreads * VEC; c += kThreads) {
    if (c0 + c >= N) continue;
    float t = red[0][c];
#pragma unroll
    for (int i = 1; i < kRowLanes; ++i) t += red[i][c];
    sums[chunk * N + c0 + c] = t;
  }
}

__global__ __launch_bounds__(kThreads)
void column_sum_kernel(const float* __restrict__ part, float* __restrict__ out, int chunks, int64_t N) {
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= N) return;
  float t = part[c];
  int i = 1;
  for (; i + 8 <= chunks; i += 8) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = part[(int64_t)(i + j) * N + c];
#pragma unroll
    for (int j = 0; j < 8; ++j) t += v[j];
  }
  for (; i < chunks; ++i) t += part[(int64_t)i * N + c];
  out[c] = t;
}

// The gated pair's: flat over 8 elements a thread where N is a multiple of 8
// (the arrays are contiguous), else one element a thread with the padded
// copies at their own row stride.
template <int ACT, int VEC>
__global__ __launch_bounds__(kThreads)
void glu_backward_kernel(const uint16_t* __restrict__ dh, const uint16_t* __restrict__ g,
                         const uint16_t* __restrict__ u, uint16_t* __restrict__ dg,
                         uint16_t* __restrict__ du, uint16_t* __restrict__ pad_g,
                         uint16_t* __restrict__ pad_u, int64_t ld, int64_t M, int64_t N) {
  const int64_t total = VEC == 1 ? M * ld : M * N;
  for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * VEC; i < total;
       i += (int64_t)gridDim.x * kThreads * VEC) {
    int64_t at = i;
    if constexpr (VEC == 1) {
      // over the padded rows: columns past N only write the copies' padding
      const int64_t r = i / ld, c = i - r * ld;
      if (c >= N) {
        if (pad_g) pad_g[i] = pad_u[i] = 0;
        continue;
      }
      at = r * N + c;
    }
    Vec<VEC> a, b, c;
    a.load(dh + at);
    b.load(g + at);
    c.load(u + at);
    float eg[VEC], eu[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float d = a.get(j), t = b.get(j);
      eg[j] = d * c.get(j) * act_grad_f32<ACT>(t);
      eu[j] = d * act_f32<ACT>(t);
    }
    Vec<VEC>::store(dg + at, eg);
    Vec<VEC>::store(du + at, eu);
    if (VEC == 1 && pad_g) {
      Vec<VEC>::store(pad_g + i, eg);
      Vec<VEC>::store(pad_u + i, eu);
    }
  }
}

__global__ __launch_bounds__(kThreads)
void fill_zero_kernel(uint32_t* __restrict__ p, size_t words, uint16_t* __restrict__ tail) {
  for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < words; i += (size_t)gridDim.x * kThreads)
    p[i] = 0;
  if (tail && blockIdx.x == 0 && threadIdx.x == 0) *tail = 0;
}

constexpr int64_t kMaxBlocks = 1 << 22;   // threads of a launch stay below 2^32

int64_t column_blocks(int64_t n, int vec) { return (n + kColThreads * vec - 1) / (kColThreads * vec); }

// Rows per chunk: enough workgroups to fill the GPU (about eight a CU), at
// most 256 chunks, and at least 128 rows in one, so that a short call needs no
// second kernel for its column sums.
int64_t chunk_rows(int64_t m, int64_t n) {
  const int64_t cols = column_blocks(n, n % 8 == 0 ? 8 : 1);
  int64_t chunks = (2048 + cols - 1) / cols;
  if (chunks > 256) chunks = 256;
  int64_t rows = (m + chunks - 1) / chunks;
  return rows < 128 ? 128 : rows;
}

}  // namespace

size_t column_sum_bytes(int64_t m, int64_t n) {
  const int64_t rows = chunk_rows(m, n);
  const int64_t chunks = (m + rows - 1) / rows;
  return chunks > 1 ? round_up((size_t)(chunks * n) * 4, kWorkspaceAlign) : 0;
}

hipError_t launch_act_backward(const uint16_t* dy, const uint16_t* z, uint16_t* dz, uint16_t* pad,
                               int64_t ld, float* dbias, float* part, int64_t m, int64_t n, int act,
                               hipStream_t stream) {
  const int64_t rows = chunk_rows(m, n);
  const int64_t chunks = (m + rows - 1) / rows;
  float* sums = dbias == nullptr ? nullptr : chunks > 1 ? part : dbias;
  const bool wide = n % 8 == 0;
  // the narrow form also covers the padding columns
  const int64_t cols = wide ? column_blocks(n, 8) : column_blocks(pad ? ld : n, 1);
  const dim3 grid((uint32_t)(cols * chunks));
  with_act(act, [&](auto a) {
    constexpr int A = decltype(a)::value;
    if (wide)
      hipLaunchKernelGGL((act_backward_kernel<A, 8>), grid, dim3(kThreads), 0, stream, dy, z, dz, pad,
                         ld, sums, m, n, rows, (int)cols);
    else
      hipLaunchKernelGGL((act_backward_kernel<A, 1>), grid, dim3(kThreads), 0, stream, dy, z, dz, pad,
                         ld, sums, m, n, rows, (int)cols);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || dbias == nullptr || chunks == 1) return e;
  hipLaunchKernelGGL(column_sum_kernel, dim3((uint32_t)((n + kThreads - 1) / kThreads)), dim3(kThreads),
                     0, stream, part, dbias, (int)chunks, n);
  return hipGetLastError();
}

hipError_t launch_glu_backward(const uint16_t* dh, const uint16_t* g, const uint16_t* u, uint16_t* dg,
                               uint16_t* du, uint16_t* pad_g, uint16_t* pad_u, int64_t ld, int64_t m,
                               int64_t n, int act, hipStream_t stream) {
  const bool wide = n % 8 == 0;
  const int64_t blocks = ((wide ? m * n / 8 : m * ld) + kThreads - 1) / kThreads;
  const dim3 grid((uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks));
  with_act(act, [&](auto a) {
    constexpr int A = decltype(a)::value;
    if (wide)
      hipLaunchKernelGGL((glu_backward_kernel<A, 8>), grid, dim3(kThreads), 0, stream, dh, g, u, dg, du,
                         pad_g, pad_u, ld, m, n);
    else
      hipLaunchKernelGGL((glu_backward_kernel<A, 1>), grid, dim3(kThreads), 0, stream, dh, g, u, dg, du,
                         pad_g, pad_u, ld, m, n);
  });
  return hipGetLastError();
}

hipError_t launch_fill_zero(void* p, size_t bytes, hipStream_t stream) {
  const size_t words = bytes / 4;
  const size_t want = (words + kThreads - 1) / kThreads;
  const uint32_t blocks = (uint32_t)(want < 1 ? 1 : want > 4096 ? 4096 : want);
  uint16_t* tail = (bytes & 2) ? reinterpret_cast<uint16_t*>(static_cast<char*>(p) + words * 4) : nullptr;
  hipLaunchKernelGGL(fill_zero_kernel, dim3(blocks), dim3(kThreads), 0, stream,
                     static_cast<uint32_t*>(p), words, tail);
  return hipGetLastError();
}

}  // namespace fp8bl
