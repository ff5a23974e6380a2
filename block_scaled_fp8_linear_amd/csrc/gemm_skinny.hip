// Skinny-M block-FP8 linear (M <= 32 per pass): the run is bound by the HBM
// bytes of the E4M3 weight, so the kernel is organised around streaming W
// once, at full bandwidth.
//
// Same arithmetic as the tiled path (FastVideo PR #1829, "Purpose": the
// weight goes to BF16, then an ordinary matmul; fp32 accumulation, one bf16
// rounding per output).
//
// Work unit: a workgroup of W waves owns 32 weight rows (two 16-row tiles)
// and one K range (its split; normally all of K). The range is cut into
// 256-wide super-steps dealt round-robin to the waves.
//
// Load shape. HBM streams well when each load instruction reads a few long
// runs: 4 rows x 256 contiguous bytes per 64-lane instruction reaches ~95%
// of a plain sequential read on MI355X, while the MFMA operand shape (16
// rows x 64 bytes) reaches ~60%. So codes are loaded 4 rows x 256 bytes at a
// time straight into a per-wave LDS slab (16-byte buffer loads that write
// LDS: lane i lands at byte 16*i of the instruction's 1 KB, and fetches the
// 16-byte chunk that puts each row's chunks XOR-permuted by the row index,
// so the MFMA-layout reads back are bank-conflict-free). No barrier is
// needed because each wave only reads what it loaded. Rows past N and the K
// tail read as zero through the buffer descriptors.
//
// The k order inside a super-step is permuted (the MFMA sums over k, so A
// and B only have to agree): MFMA 2h+e gives lane group g the codes
// k = 16*(g + 4h) + 8e .. +8, and X is loaded into registers with the same
// k. X (rows past M read as zero) is tiny and stays in L2; the two tiles of
// a wave share each X fragment. At the end the waves' partial sums meet in
// LDS and are added in wave order; with one split the result is rounded to
// bf16 directly, otherwise fp32 partials go to the workspace and are summed
// in split order by the reduce kernel (no atomics anywhere).
//
// v_mfma_f32_16x16x32_bf16: lane l gives 8 consecutive-k values of row
// (l % 16) of A and of column (l % 16) of B; lane group l / 16 picks the
// k chunk. Output: lane l holds rows (l/16)*4 + r, r = 0..3, column l % 16.
#include "gemm_skinny_body.h"

namespace fp8bl {

namespace {

template <int MT, int NT, int WAVES, int D>
__global__ __launch_bounds__(WAVES * 64)
void gemm_skinny_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ q,
                        const float* __restrict__ s, uint16_t* __restrict__ y,
                        float* __restrict__ part, int M, int N, int K, int gk,
                        int ss_per_split) {
  gemm_skinny_body<MT, NT, WAVES, D, kSkinnyPlain>(x, q, s, nullptr, nullptr, y, part, M, N, K, gk,
                                                   ss_per_split, LayerEpilogue{});
}

// Sum of split-K partials, 8 outputs per thread (two 16-byte loads per
// split), added in split order and rounded once; a scalar tail handles
// M*N not divisible by 8. With the split count fixed at compile time every
// load is in flight before the first add (bit-identical; 1-5% faster than
// the run-time loop on MI355X, which waits for each split's loads in turn).
// S > 0: exactly S splits, every load issued before the first add; S == 0:
// `splits` at run time.
template <int S>
__global__ __launch_bounds__(256)
void reduce_partials_kernel(const float* __restrict__ part, uint16_t* __restrict__ y,
                            int splits, size_t mn, size_t slab) {
  const size_t i8 = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if constexpr (S == 0) {
    if (i8 + 8 <= mn) {
      f32x4 a = *reinterpret_cast<const f32x4*>(part + i8);
      f32x4 b = *reinterpret_cast<const f32x4*>(part + i8 + 4);
      for (int sp = 1; sp < splits; ++sp) {
        const f32x4 c = *reinterpret_cast<const f32x4*>(part + (size_t)sp * slab + i8);
        const f32x4 d = *reinterpret_cast<const f32x4*>(part + (size_t)sp * slab + i8 + 4);
        a[0] += c[0]; a[1] += c[1]; a[2] += c[2]; a[3] += c[3];
        b[0] += d[0]; b[1] += d[1]; b[2] += d[2]; b[3] += d[3];
      }
      u32x4 o = {pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                 pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
      *reinterpret_cast<u32x4*>(y + i8) = o;
      return;
    }
  } else if (i8 + 8 <= mn) {
    f32x4 c[S], d[S];
#pragma unroll
    for (int sp = 0; sp < S; ++sp) {
      c[sp] = *reinterpret_cast<const f32x4*>(part + (size_t)sp * slab + i8);
      d[sp] = *reinterpret_cast<const f32x4*>(part + (size_t)sp * slab + i8 + 4);
    }
    f32x4 a = c[0], b = d[0];
#pragma unroll
    for (int sp = 1; sp < S; ++sp) {
      a[0] += c[sp][0]; a[1] += c[sp][1]; a[2] += c[sp][2]; a[3] += c[sp][3];
      b[0] += d[sp][0]; b[1] += d[sp][1]; b[2] += d[sp][2]; b[3] += d[sp][3];
    }
    u32x4 o = {pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
               pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
    *reinterpret_cast<u32x4*>(y + i8) = o;
    return;
  }
  if (i8 < mn) {
    for (size_t i = i8; i < mn; ++i) {
      float t = part[i];
      for (int sp = 1; sp < (S > 0 ? S : splits); ++sp) t += part[(size_t)sp * slab + i];
      const __bf16 v = (__bf16)t;
      y[i] = __builtin_bit_cast(uint16_t, v);
    }
  }
}

}  // namespace

// From measurements on MI355X (N=8000, K=8192): 4 waves per workgroup and
// 32 weight rows per workgroup (two 16-row tiles sharing each X fragment)
// for every M; 16 rows per workgroup, twice the workgroups, were 6% slower
// even at M = 1.
SkinnyPlan plan_skinny(int64_t m, int64_t n, int64_t k) {
  SkinnyPlan p;
  p.mt = m > 16 ? 2 : 1;
  p.nt = 2;
  const int nss = (int)((k + kSuper - 1) / kSuper);
  const int64_t groups = (n + 16 * p.nt - 1) / (16 * p.nt);
  int splits = 1;
  // Split K only when there are too few row groups to occupy the GPU,
  // keeping >= 2 super-steps per wave.
  while (groups * splits < 192 && nss / (splits * 2) >= kWaves * 2) splits *= 2;
  p.ss_per_split = (nss + splits - 1) / splits;
  p.splits = (nss + p.ss_per_split - 1) / p.ss_per_split;
  return p;
}

hipError_t launch_reduce_partials(const float* part, uint16_t* y, int splits,
                                  int64_t m, int64_t n, hipStream_t stream) {
  const size_t mn = (size_t)m * (size_t)n;
  const size_t blocks = (mn + 256 * 8 - 1) / (256 * 8);
  const size_t slab = partial_slab((size_t)m, (size_t)n);
  const dim3 grid((uint32_t)blocks);
  switch (splits) {
    case 2: hipLaunchKernelGGL(reduce_partials_kernel<2>, grid, dim3(256), 0, stream, part, y, splits, mn, slab); break;
    case 3: hipLaunchKernelGGL(reduce_partials_kernel<3>, grid, dim3(256), 0, stream, part, y, splits, mn, slab); break;
    case 4: hipLaunchKernelGGL(reduce_partials_kernel<4>, grid, dim3(256), 0, stream, part, y, splits, mn, slab); break;
    case 5: hipLaunchKernelGGL(reduce_partials_kernel<5>, grid, dim3(256), 0, stream, part, y, splits, mn, slab); break;
    case 6: hipLaunchKernelGGL(reduce_partials_kernel<6>, grid, dim3(256), 0, stream, part, y, splits, mn, slab); break;
    case 7: hipLaunchKernelGGL(reduce_partials_kernel<7>, grid, dim3(256), 0, stream, part, y, splits, mn, slab); break;
    case 8: hipLaunchKernelGGL(reduce_partials_kernel<8>, grid, dim3(256), 0, stream, part, y, splits, mn, slab); break;
    default: hipLaunchKernelGGL(reduce_partials_kernel<0>, grid, dim3(256), 0, stream, part, y, splits, mn, slab);
  }
  return hipGetLastError();
}

size_t skinny_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  // Passes of up to 32 rows of X run one after another through the same
  // workspace; size for the widest pass.
  const int64_t rows = m < 32 ? m : 32;
  if (rows == 0) return 0;
  const SkinnyPlan p = plan_skinny(rows, n, k);
  if (p.splits <= 1) return 0;
  return round_up((size_t)p.splits * partial_slab(rows, n) * sizeof(float), kWorkspaceAlign);
}

hipError_t launch_gemm_skinny(const uint16_t* x, const uint8_t* q, const float* s,
                              uint16_t* y, int64_t m, int64_t n, int64_t k,
                              void* ws, size_t ws_bytes, hipStream_t stream) {
  const int gk = (int)((k + kBlock - 1) / kBlock);
  for (int64_t r0 = 0; r0 < m; r0 += 32) {
    const int64_t rows = (m - r0) < 32 ? (m - r0) : 32;
    const SkinnyPlan p = plan_skinny(rows, n, k);
    float* part = p.splits > 1 ? static_cast<float*>(ws) : nullptr;
    if (p.splits > 1 && (ws == nullptr || ws_bytes < (size_t)p.splits * partial_slab(rows, n) * sizeof(float)))
      return hipErrorInvalidValue;
    const dim3 grid((uint32_t)((n + 16 * p.nt - 1) / (16 * p.nt)), (uint32_t)p.splits);
    const uint16_t* xp = x + (size_t)r0 * k;
    uint16_t* yp = y + (size_t)r0 * n;
    const dim3 block(kWaves * 64);
    if (p.mt == 1)
      hipLaunchKernelGGL((gemm_skinny_kernel<1, 2, kWaves, kRing>), grid, block, 0, stream, xp, q,
                         s, yp, part, (int)rows, (int)n, (int)k, gk, p.ss_per_split);
    else
      hipLaunchKernelGGL((gemm_skinny_kernel<2, 2, kWaves, kRing>), grid, block, 0, stream, xp, q,
                         s, yp, part, (int)rows, (int)n, (int)k, gk, p.ss_per_split);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.splits > 1) {
      e = launch_reduce_partials(part, yp, p.splits, rows, n, stream);
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace fp8bl
