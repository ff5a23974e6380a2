// Elementwise part of the layer operators' backward passes, bound by HBM.
//
//   linear: dz = dy act'(z), dbias[c] = sum over rows of dz[r, c]
//   gated:  dg = dh u act'(g), du = dh act(g)
//
// A thread handles eight consecutive columns of a row. Where N is no multiple
// of 8 rows start at any 2-byte address: the accesses stay 16 bytes wide (the
// hardware takes global ones at any alignment), the last columns of a row go
// one by one, and the kernels also write a copy with padded rows (`ld`
// elements, the padding zero), which is what the product that follows reads
// in whole 16-byte chunks. (4096 x 12288 with GELU and the column sums 57 us
// and 5 for their join, 5.3 TB/s; the gated pair at 4096 x 12800 83 us, 6.3
// TB/s; odd rows, 809 x 8449 with GELU and sums, 13 us against 23 with one
// element a thread.)
#include "fp8bl_act.h"
#include "fp8bl_device.h"
#include "fp8bl_internal.h"

namespace fp8bl {

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;

// Eight columns of a row from `col`, or the `left` < 8 that exist (the others
// read as zero and are not written).
__device__ __forceinline__ void load8(const uint16_t* p, int left, float (&f)[kVec]) {
  if (left >= kVec) {
    u32x4 v;
    __builtin_memcpy(&v, p, 16);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      f[i] = __uint_as_float((i & 1) ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = i < left ? bf16_f32(p[i]) : 0.0f;
  }
}
__device__ __forceinline__ u32x4 pack8(const float (&f)[kVec]) {
  return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
               pack_bf16x2(f[6], f[7])};
}
__device__ __forceinline__ void store8(uint16_t* p, int left, const float (&f)[kVec]) {
  if (left >= kVec) {
    const u32x4 v = pack8(f);
    __builtin_memcpy(p, &v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i < left) p[i] = f32_bf16(f[i]);
  }
}

// A workgroup of CT threads along a row and 256 / CT rows covers 8 CT columns
// and one chunk of rows: thread (rl, cl) takes rows rl, rl + 256 / CT, ... of
// the chunk. The column sums of the row lanes meet in LDS and are added in
// lane order; the chunks' sums go to `sums` [chunks, N] and are added in order
// by the second kernel (no atomics: the same bits on every call). dz may be
// null (act none: dz is dy), the padded copy and the sums too.
template <int ACT, int CT>
__global__ __launch_bounds__(kThreads)
void act_backward_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ z,
                         uint16_t* __restrict__ dz, uint16_t* __restrict__ pad, int64_t ld,
                         float* __restrict__ sums, int64_t M, int64_t N, int64_t rows_per_chunk,
                         int col_blocks) {
  constexpr int kRowLanes = kThreads / CT;
  __shared__ float red[kRowLanes][kVec][CT + 1];
  const int cl = threadIdx.x % CT, rl = threadIdx.x / CT;
  const int64_t chunk = blockIdx.x / (uint32_t)col_blocks;
  const int64_t c0 = (int64_t)(blockIdx.x % (uint32_t)col_blocks) * CT * kVec;
  const int64_t col = c0 + cl * kVec;
  const int64_t r1 = min((chunk + 1) * rows_per_chunk, M);
  const int left = (int)min(N - col, (int64_t)kVec);
  float sum[kVec] = {};
  // whole chunks and a row's last columns in loops of their own: no branch
  // between the loads of several rows
  auto rows = [&](auto full) {
    const int n8 = decltype(full)::value ? kVec : left;
#pragma unroll 2
    for (int64_t r = chunk * rows_per_chunk + rl; r < r1; r += kRowLanes) {
      float d[kVec], t[kVec];
      load8(dy + r * N + col, n8, d);
      if constexpr (ACT != kActNone) {
        load8(z + r * N + col, n8, t);
#pragma unroll
        for (int i = 0; i < kVec; ++i) d[i] *= act_grad_f32<ACT>(t[i]);
        if (dz) store8(dz + r * N + col, n8, d);
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) sum[i] += d[i];
      // (columns past N hold zero: 0 from load8 times a finite derivative)
      if (pad) *reinterpret_cast<u32x4*>(pad + r * ld + col) = pack8(d);
    }
  };
  if (left >= kVec)
    rows(ActTag<1>{});
  else if (left > 0)
    rows(ActTag<0>{});
  if (!sums) return;
#pragma unroll
  for (int i = 0; i < kVec; ++i) red[rl][i][cl] = sum[i];
  __syncthreads();
  const int c = threadIdx.x;
  static_assert(CT * kVec <= kThreads, "one column a thread");
  if (c >= CT * kVec || c0 + c >= N) return;
  float t = red[0][c % kVec][c / kVec];
#pragma unroll
  for (int i = 1; i < kRowLanes; ++i) t += red[i][c % kVec][c / kVec];
  sums[chunk * N + c0 + c] = t;
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

// The gated pair's: one 8-column chunk of a row a thread, `chunks` to a row,
// grid-stride (where N is a multiple of 8 the chunks of all rows are
// contiguous).
template <int ACT>
__global__ __launch_bounds__(kThreads)
void glu_backward_kernel(const uint16_t* __restrict__ dh, const uint16_t* __restrict__ g,
                         const uint16_t* __restrict__ u, uint16_t* __restrict__ dg,
                         uint16_t* __restrict__ du, uint16_t* __restrict__ pad_g,
                         uint16_t* __restrict__ pad_u, int64_t M, int64_t N, int64_t chunks) {
  const int64_t total = M * chunks;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    int64_t at = i * kVec;
    int left = kVec;
    if (pad_g || chunks * kVec != N) {
      const int64_t r = i / chunks, col = (i - r * chunks) * kVec;
      at = r * N + col;
      left = (int)min(N - col, (int64_t)kVec);
    }
    float a[kVec], b[kVec], c[kVec], eg[kVec], eu[kVec];
    load8(dh + at, left, a);
    load8(g + at, left, b);
    load8(u + at, left, c);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      eg[j] = a[j] * c[j] * act_grad_f32<ACT>(b[j]);
      eu[j] = a[j] * act_f32<ACT>(b[j]);
    }
    store8(dg + at, left, eg);
    store8(du + at, left, eu);
    if (pad_g) {
      *reinterpret_cast<u32x4*>(pad_g + i * kVec) = pack8(eg);
      *reinterpret_cast<u32x4*>(pad_u + i * kVec) = pack8(eu);
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

// Up to 256 rows narrow workgroups (8 threads along a row) take all rows as
// one chunk, so that a short call needs no second kernel for its column sums
// and still has workgroups enough; else wide ones (32 threads), about eight a
// CU, with at least 32 rows in a chunk and at most 256 chunks. (77 x 1003 with
// SiLU and sums: 6.4 us; as four wide workgroups 18.)
struct RowPlan {
  int ct;
  int64_t rows, chunks;
};
int64_t column_blocks(int64_t n, int ct) { return (n + ct * kVec - 1) / (ct * kVec); }
RowPlan plan_rows(int64_t m, int64_t n) {
  if (m <= 256) return RowPlan{8, 256, 1};
  int64_t chunks = (2048 + column_blocks(n, 32) - 1) / column_blocks(n, 32);
  if (chunks > 256) chunks = 256;
  int64_t rows = (m + chunks - 1) / chunks;
  rows = rows < 32 ? 32 : rows;
  return RowPlan{32, rows, (m + rows - 1) / rows};
}

}  // namespace

size_t column_sum_bytes(int64_t m, int64_t n) {
  const int64_t chunks = plan_rows(m, n).chunks;
  return chunks > 1 ? round_up((size_t)(chunks * n) * 4, kWorkspaceAlign) : 0;
}

hipError_t launch_act_backward(const uint16_t* dy, const uint16_t* z, uint16_t* dz, uint16_t* pad,
                               int64_t ld, float* dbias, float* part, int64_t m, int64_t n, int act,
                               hipStream_t stream) {
  const RowPlan p = plan_rows(m, n);
  const int64_t chunks = p.chunks;
  float* sums = dbias == nullptr ? nullptr : chunks > 1 ? part : dbias;
  const int64_t cols = column_blocks(n, p.ct);
  const dim3 grid((uint32_t)(cols * chunks));
  with_act(act, [&](auto a) {
    constexpr int A = decltype(a)::value;
    if (p.ct == 8)
      hipLaunchKernelGGL((act_backward_kernel<A, 8>), grid, dim3(kThreads), 0, stream, dy, z, dz, pad, ld, sums, m,
                         n, p.rows, (int)cols);
    else
      hipLaunchKernelGGL((act_backward_kernel<A, 32>), grid, dim3(kThreads), 0, stream, dy, z, dz, pad, ld, sums,
                         m, n, p.rows, (int)cols);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || dbias == nullptr || chunks == 1) return e;
  hipLaunchKernelGGL(column_sum_kernel, dim3((uint32_t)((n + kThreads - 1) / kThreads)), dim3(kThreads),
                     0, stream, part, dbias, (int)chunks, n);
  return hipGetLastError();
}

hipError_t launch_glu_backward(const uint16_t* dh, const uint16_t* g, const uint16_t* u, uint16_t* dg,
                               uint16_t* du, uint16_t* pad_g, uint16_t* pad_u, int64_t m, int64_t n, int act,
                               hipStream_t stream) {
  const int64_t chunks = (n + kVec - 1) / kVec;        // ld / 8 where there are padded copies
  const int64_t blocks = (m * chunks + kThreads - 1) / kThreads;
  const dim3 grid((uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks));
  with_act(act, [&](auto a) {
    hipLaunchKernelGGL((glu_backward_kernel<decltype(a)::value>), grid, dim3(kThreads), 0, stream, dh, g, u, dg,
                       du, pad_g, pad_u, m, n, chunks);
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
