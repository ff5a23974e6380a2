// Fused block-FP8 linear for large M: Y[M,N] = X[M,K] * W_hat[N,K]^T, with
// W_hat = bf16(fl32(e4m3(Q) * S)) formed in registers only (FastVideo PR
// #1829, "Purpose": block-scaled weight to BF16, then an ordinary matmul;
// LightX2V PR #1657, "Walkthrough": FP32 accumulation).
//
// Tile 256 (X rows) x 256 (weight rows), one workgroup of four waves per CU.
// Wave w owns weight rows [64w, 64w + 64) of the tile against all 256 X
// rows: 2 x 8 blocks of v_mfma_f32_32x32x16_bf16, 256 fp32 accumulators per
// lane. The decoded weight is the MFMA A operand and X the B operand, so a
// lane's accumulators hold four consecutive output columns of one output
// row (the epilogue regroups them through LDS into whole-line stores). Per 64-wide K step a wave reads 32 X fragments from
// LDS, and each fragment feeds both of its weight blocks: half the LDS
// traffic per MFMA of a one-block-per-wave layout. Every code is decoded
// once per workgroup, by the wave that owns its row.
//
// Data movement per step, through a ring of three LDS stages:
//  - X: 32 KB per stage, moved global -> LDS by 16-byte buffer loads that
//    write LDS directly (no registers). The 16-byte chunks of a 128-byte LDS
//    row are XOR-permuted by (row / 2) % 8, chosen on the global side, so
//    that the MFMA operand reads (16 lanes on 16 consecutive rows, one
//    chunk) hit 16 distinct bank groups.
//  - codes: 16 KB per stage, moved the same way (each wave loads only the 64
//    rows it decodes, 16 rows x 64 bytes per instruction), the 16-byte
//    chunks of a row XOR-permuted by (row / 4) % 4 so the decoding reads are
//    conflict-free.
//  - weight scale: one word per wave and step, moved into the stage the
//    same way, so that no global load in the main loop writes a register and
//    the compiler adds no waits of its own on them.
//  - the 13 loads of a wave's share of a stage go out two steps ahead,
//    spread over the first three quarters of a step (one per four MFMAs).
//    Issued in one burst after the barrier, as four waves at once, they
//    filled the CU's load queue and held the MFMA stream behind it.
//
// Register pipeline inside a step (four sub-steps of k16, 64 MFMAs): X
// fragments are read from LDS four ahead of their MFMAs into a ring of
// eight registers; sub-step t+1's weight operands are decoded during
// sub-step t (E4M3 -> fp32 convert, one fp32 multiply by the scale, RNE to
// bf16), the next step's first ones during the last two quarter-sub-steps.
// The step runs as 16 regions of 4 MFMAs, each with its own share of the
// reads, the decode and the loads, in a fixed order (a scheduling barrier
// between regions keeps the compiler from pairing an MFMA with a read it
// has just issued). One barrier per step, 8 MFMAs before its end.
//
// The K order inside a step is a permutation (A and B only have to agree):
// lane half h holds, for sub-step t, k = 16h + 32(t/2) + 8(t%2) .. +8, so a
// lane's codes for the step are two contiguous 16-byte runs of its row.
//
// Rows past M or N and K past the end read as zero through buffer
// descriptors that cover only valid rows and through per-lane out-of-range
// offsets; no branch in the main loop depends on data.
//
// Persistent: one workgroup per CU walks its (tile, K split) units; the
// loads of the next unit's first two steps go out during the last two steps
// of the current one, so the ring never drains between units.
//
// Split-K (units with a K split): every split writes its fp32 partial tile to
// the workspace and the ordered reduce kernel adds the splits and rounds once.
//
// Gated (the MLP gate/up pair with the SwiGLU epilogue): the tile covers 128
// output columns; waves 0 and 1 run its gate weight rows and waves 2 and 3
// the same rows of the up weight, everything else as above. Wave w and wave
// w + 2 then hold the two products of one 256 x 64 output slice, element for
// element, and finish half of it each after trading the other half through
// LDS.
#include <atomic>

#include "gemm_large_body.h"

namespace fp8bl {

namespace {

template <bool SPLIT, bool GATED>
__global__ __launch_bounds__(kThreads, 1)
void gemm_large_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ q,
                       const float* __restrict__ s, const uint8_t* __restrict__ q2,
                       const float* __restrict__ s2, uint16_t* __restrict__ y,
                       float* __restrict__ part, int M, int N, int K, int gk,
                       int tiles_m, int tiles_n, int kt_per_split, int splits, int steps_per_unit) {
  gemm_large_body<SPLIT, GATED, kPlain, kActNone>(x, q, s, q2, s2, y, part, M, N, K, gk, tiles_m, tiles_n,
                                                  kt_per_split, splits, steps_per_unit, LargeArgs{});
}

}  // namespace

// Split count from the cost model of the tile-planned kernel's planner, in
// the same units (microseconds, work counted in 128x128x64 steps): a CU
// runs this kernel's 256x256x64 step (4 of those) at 2.42 of them per
// microsecond (measured on 16384 x 12288 x 3072), plus about 2 us per unit
// for its first loads and its epilogue; the busiest CU sets the time, ceil(units /
// 256) units. K splits add the fp32 partials' round trip (as in that
// planner). The split count that puts about one unit on every CU wins at
// 512 rows (e.g. 6 for 512 x 5120 x 25600).
LargePlan plan_large(int64_t m, int64_t n, int64_t k) {
  const int nkt = (int)((k + kBK - 1) / kBK);
  const int64_t tiles = ((m + kBM - 1) / kBM) * ((n + kBN - 1) / kBN);
  LargePlan p{1, nkt, 0.0};
  double best = 1e300;
  for (int sp = 1; sp <= 8; ++sp) {
    const int steps = (nkt + sp - 1) / sp;
    if (sp > 1 && steps < 8) break;
    const int64_t per_cu = (tiles * sp + 255) / 256;
    double cost = (double)per_cu * (steps * 4 / 2.42 + 2.0);
    if (sp > 1) cost += (double)(6 * sp + 2) * (double)(m * n) / 5.0e6;
    if (cost < best) {
      best = cost;
      p.splits = sp;
    }
  }
  p.kt_per_split = (nkt + p.splits - 1) / p.splits;
  p.splits = (nkt + p.kt_per_split - 1) / p.kt_per_split;
  p.cost = best;
  return p;
}

size_t large_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  const LargePlan p = plan_large(m, n, k);
  if (p.splits <= 1) return 0;
  return round_up((size_t)p.splits * partial_slab(m, n) * sizeof(float), kWorkspaceAlign);
}

// Compute units of the current device (persistent grid size), cached.
namespace {
constexpr int kMaxDev = 64;
std::atomic<int> g_cus[kMaxDev];
}  // namespace

int device_cus() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDev) return 256;
  int v = g_cus[dev].load(std::memory_order_relaxed);
  if (v <= 0) {
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0)
      v = 256;
    g_cus[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

hipError_t launch_gemm_large_partials(const LargePlan& p, const uint16_t* x, const uint8_t* q,
                                      const float* s, float* part, int64_t m, int64_t n, int64_t k,
                                      hipStream_t stream) {
  const int tiles_m = (int)((m + kBM - 1) / kBM);
  const int tiles_n = (int)((n + kBN - 1) / kBN);
  const int units = tiles_m * tiles_n * p.splits;
  const int grid = units < device_cus() ? units : device_cus();
  const int spu = p.kt_per_split > 2 ? p.kt_per_split : 2;
  hipLaunchKernelGGL((gemm_large_kernel<true, false>), dim3((uint32_t)grid), dim3(kThreads), 0,
                     stream, x, q, s, nullptr, nullptr, nullptr, part, (int)m, (int)n, (int)k,
                     (int)((k + kBlock - 1) / kBlock), tiles_m, tiles_n, p.kt_per_split, p.splits, spu);
  return hipGetLastError();
}

hipError_t launch_gemm_large(const uint16_t* x, const uint8_t* q, const float* s, uint16_t* y,
                             int64_t m, int64_t n, int64_t k, void* ws, size_t ws_bytes,
                             hipStream_t stream) {
  const LargePlan p = plan_large(m, n, k);
  const int gk = (int)((k + kBlock - 1) / kBlock);
  const int tiles_m = (int)((m + kBM - 1) / kBM);
  const int tiles_n = (int)((n + kBN - 1) / kBN);
  if (p.splits == 1) {
    // one persistent workgroup per CU; every unit has at least two steps (the
    // prologue loads two; a padded step reads zeros)
    const int units = tiles_m * tiles_n;
    const int grid = units < device_cus() ? units : device_cus();
    const int spu = p.kt_per_split > 2 ? p.kt_per_split : 2;
    hipLaunchKernelGGL((gemm_large_kernel<false, false>), dim3((uint32_t)grid), dim3(kThreads), 0,
                       stream, x, q, s, nullptr, nullptr, y, nullptr, (int)m, (int)n, (int)k, gk,
                       tiles_m, tiles_n, p.kt_per_split, 1, spu);
    return hipGetLastError();
  }
  if (ws == nullptr || ws_bytes < large_workspace_bytes(m, n, k)) return hipErrorInvalidValue;
  float* part = static_cast<float*>(ws);
  hipError_t e = launch_gemm_large_partials(p, x, q, s, part, m, n, k, stream);
  if (e != hipSuccess) return e;
  return launch_reduce_partials(part, y, p.splits, m, n, stream);
}

// The gated form's tiles are 256 x 128 outputs, each the work of a plain
// 256 x 256 tile, never split: the plain model at one split, with the rate
// measured on the gate/up pair at 512 and 768 rows (2.7 steps per
// microsecond per CU; the 2.42 above is from 16384 rows, where the chip runs
// at lower clocks). Against the tiled gate/up planner it picked the faster
// kernel on all seven shapes measured (128 to 4096 rows).
double large_gated_cost(int64_t m, int64_t n, int64_t k) {
  const int nkt = (int)((k + kBK - 1) / kBK);
  const int64_t tiles = ((m + kBM - 1) / kBM) * ((n + kBN / 2 - 1) / (kBN / 2));
  return (double)((tiles + 255) / 256) * (nkt * 4 / 2.7 + 2.0);
}

hipError_t launch_gemm_large_gated(const uint16_t* x, const uint8_t* qg, const float* sg,
                                   const uint8_t* qu, const float* su, uint16_t* h, int64_t m,
                                   int64_t n, int64_t k, hipStream_t stream) {
  if ((n & 7) != 0) return hipErrorInvalidValue;
  const int nkt = (int)((k + kBK - 1) / kBK);
  const int gk = (int)((k + kBlock - 1) / kBlock);
  const int tiles_m = (int)((m + kBM - 1) / kBM);
  const int tiles_n = (int)((n + kBN / 2 - 1) / (kBN / 2));
  const int units = tiles_m * tiles_n;
  const int grid = units < device_cus() ? units : device_cus();
  const int spu = nkt > 2 ? nkt : 2;
  hipLaunchKernelGGL((gemm_large_kernel<false, true>), dim3((uint32_t)grid), dim3(kThreads), 0,
                     stream, x, qg, sg, qu, su, h, nullptr, (int)m, (int)n, (int)k, gk, tiles_m,
                     tiles_n, nkt, 1, spu);
  return hipGetLastError();
}

}  // namespace fp8bl
