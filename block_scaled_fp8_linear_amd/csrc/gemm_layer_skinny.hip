// Layer operators at few rows (M <= 32): the skinny kernel's loop with the
// epilogues, and the input gradient as a stream over the weight's rows. All
// are bound by the codes, each read once; with a small weight by the launch
// and the latency of a wave's few loads.
#include "gemm_skinny_body.h"
#include "layer_plan.h"

namespace fp8bl {

using namespace plan;

namespace {

static_assert(kStreamK == kSuper && kStreamWaves == kWaves, "the plans' streams are the kernels'");

// y = act(x W^T + bias) + residual on the sums that meet in LDS.
// (1 x 8000 x 8192 12.6 us, 5.2 TB/s of codes, partly from the last-level
// cache; 16 x 5120 x 5120 with residual 10.7 us. Eight waves where no CU has
// two workgroups, so half the iterations a wave: 9.3 against 9.1 us at 1 x
// 5120 x 5120, 15.9 against 15.0 at 1 x 8000 x 8192.)
template <typename P>
__global__ __launch_bounds__(kWaves * 64, P::kResident)
void linear_act_skinny_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ q,
                              const float* __restrict__ s, uint16_t* y, float* __restrict__ part, int M,
                              int N, int K, int gk, int ss_per_split, LayerEpilogue ep) {
  gemm_skinny_body<P::MT, 2, kWaves, P::D, kSkinnyLayer, P::kLds, P::KW>(x, q, s, nullptr, nullptr, y, part, M, N,
                                                                         K, gk, ss_per_split, ep);
}

// h = act(x Wg^T) (x Wu^T): of a workgroup's two 16-row tiles one is gate rows
// and the other the up rows of the same 16 columns, so a lane ends with both
// sums of its outputs. (1 x 25600 x 5120 43 - 47 us, 5.6 - 6.1 TB/s of codes.)
template <typename P>
__global__ __launch_bounds__(kWaves * 64, P::kResident)
void glu_skinny_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ qg,
                       const float* __restrict__ sg, const uint8_t* __restrict__ qu,
                       const float* __restrict__ su, uint16_t* h, float* __restrict__ part, int M, int N,
                       int K, int gk, int ss_per_split, LayerEpilogue ep) {
  gemm_skinny_body<P::MT, 2, kWaves, P::D, kSkinnyGlu, P::kLds, P::KW>(x, qg, sg, qu, su, h, part, M, N, K, gk,
                                                                       ss_per_split, ep);
}

// ---- Input gradient, dx[M,C] = a W (+ a2 W2), few rows: bound by the codes'
// bytes, each read once. (16 x 12288 x 4096, weight rows x columns, 17.7 us
// with the join, 2.8 TB/s; 16 x 25600 x 5120 40.5 us, 3.2 TB/s: the X rows of
// every strip and its fp32 partials are the rest.)
//
// A workgroup owns 256 output columns and a range of weight rows (its split);
// the range is cut into super-steps of 32 rows dealt round-robin to its four
// waves. A super-step's codes (32 rows x 256 bytes, 4 rows per load
// instruction as in the forward) go straight to a two-slot LDS ring of the
// wave; 16-byte chunk c of row r is stored at c ^ (r % 16). The MFMA operand
// needs eight consecutive rows of one column per lane: ds_read_b64_tr_b8
// transposes on the way out (in each group of 16 lanes, lanes 2r and 2r + 1
// address the halves of row r's 16 columns, lane i receives column i). Its 32
// lanes served together read 16 bytes of 16 rows, at 16 distinct chunks: no
// bank conflict. The left operand's eight values are one 16-byte load.
//
// v_mfma_f32_16x16x32_bf16: lane l holds row (l % 16) of the left operand and
// column (l % 16) of the right one at k = 8 (l / 16) .. +8.
constexpr int kStripTiles = kStripCols / 16;
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2* lds_i32x2_ptr_t;

template <int MT>
__global__ __launch_bounds__(kWaves * 64, 2)
void input_gradient_skinny_kernel(const uint16_t* __restrict__ a, const uint8_t* __restrict__ q,
                                  const float* __restrict__ s, const uint16_t* __restrict__ a2,
                                  const uint8_t* __restrict__ q2, const float* __restrict__ s2, int lda,
                                  uint16_t* __restrict__ dx, float* __restrict__ part, int M, int C, int R,
                                  int gk, int strips, int steps1, int steps, int steps_per_split) {
  constexpr int kSlot = kStepRows * kStripCols;
  constexpr int kLoads = 8 + MT;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kWaves][kRing][kSlot];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int strip = (int)(blockIdx.x % (uint32_t)strips), split = (int)(blockIdx.x / (uint32_t)strips);
  const int c0 = strip * kStripCols;
  const int st0 = split * steps_per_split, st1 = min(st0 + steps_per_split, steps);
  uint8_t* const wring = &ring[wave][0][0];

  const uint32_t arange = (uint32_t)(M * lda * 2);
  const __amdgpu_buffer_rsrc_t ars = make_rsrc(a, arange);
  const __amdgpu_buffer_rsrc_t ars2 = make_rsrc(a2 ? a2 : a, arange);
  const int lr = lane >> 4, lc = lane & 15;
  uint32_t woff[8];
  bool cin[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int row = 4 * r + lr, chunk = lc ^ (row & 15);
    woff[r] = (uint32_t)(row * C + chunk * 16);
    cin[r] = c0 + chunk * 16 < C;
  }
  const uint32_t aoff = (uint32_t)((lc * lda + 8 * lr) * 2);
  const uint32_t atile = (uint32_t)(16 * lda * 2);

  f32x4 acc[kStripTiles][MT];
#pragma unroll
  for (int t = 0; t < kStripTiles; ++t)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto row_of = [&](int st) { return (st >= steps1 ? st - steps1 : st) * kStepRows; };
  auto issue = [&](int st, int slot, u32x4 (&xa)[MT]) {
    const bool live = st < st1, sec = st >= steps1;
    const int r0 = row_of(st);
    const int rows = live ? min(R - r0, kStepRows) : 0;
    const bool ain = 8 * lr < rows;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const uint32_t o = ain ? aoff + (uint32_t)i * atile + (uint32_t)(r0 * 2) : kOob;
      xa[i] = sec ? buf_load16(ars2, o) : buf_load16(ars, o);
    }
    const __amdgpu_buffer_rsrc_t wrs = make_rsrc(
        (sec ? q2 : q) + (live ? (size_t)r0 * C + c0 : 0),
        (uint32_t)__builtin_amdgcn_readfirstlane(rows > 0 ? rows * C - c0 : 0));
    uint8_t* const base = wring + slot * kSlot;
#pragma unroll
    for (int r = 0; r < 8; ++r)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wrs, (lds_ptr_t)(base + r * 1024), 16, cin[r] ? woff[r] : kOob,
                                               0, 0, kNonTemporal);
  };
  const int i16 = lane & 15, grp = lane >> 4;
  const int trow = 8 * grp + (i16 >> 1);
  const int tbase = trow * kStripCols + 8 * (i16 & 1);
  const int tswz = trow & 15;
  auto compute = [&](int st, int slot, const u32x4 (&xa)[MT], f32x4 (&ac)[kStripTiles][MT]) {
    const int rb = row_of(st) / kBlock;
    const float* const sr = (st >= steps1 ? s2 : s) + (size_t)rb * gk;
    const int cb = c0 / kBlock;
    const float s0 = sr[cb], s1 = cb + 1 < gk ? sr[cb + 1] : 0.0f;
    const uint8_t* const base = wring + slot * kSlot + tbase;
#pragma unroll
    for (int t = 0; t < kStripTiles; ++t) {
      const i32x2 c = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2_ptr_t)(base + ((t ^ tswz) << 4)));
      const bf16x8 b = dequant8((uint32_t)c[0], (uint32_t)c[1], t < kStripTiles / 2 ? s0 : s1);
#pragma unroll
      for (int i = 0; i < MT; ++i)
        ac[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xa[i]), b, ac[t][i], 0, 0, 0);
    }
  };

  // The same pipeline as the forward's: iteration i computes super-step
  // st0 + wave + 4 i while the next one's loads are in flight; every
  // super-step issues kLoads loads (past the range they read zero).
  const int count = st1 - st0;
  const int iters = count > wave ? (count - wave + kWaves - 1) / kWaves : 0;
  auto st_of = [&](int i) { return st0 + wave + i * kWaves; };
  u32x4 xv[2][MT];
  issue(iters > 0 ? st_of(0) : st1, 0, xv[0]);
  int i0 = 0;
  for (; i0 + 2 <= iters; i0 += 2) {
    __builtin_amdgcn_s_waitcnt(kLgkmWait0);        // the slot's reads have returned
    issue(st_of(i0 + 1), 1, xv[1]);
    __builtin_amdgcn_s_waitcnt(vm_wait(kLoads));
    compute(st_of(i0), 0, xv[0], acc);
    __builtin_amdgcn_s_waitcnt(kLgkmWait0);        // the slot's reads have returned
    issue(i0 + 2 < iters ? st_of(i0 + 2) : st1, 0, xv[0]);
    __builtin_amdgcn_s_waitcnt(vm_wait(kLoads));
    compute(st_of(i0 + 1), 1, xv[1], acc);
  }
  __builtin_amdgcn_s_waitcnt(vm_wait(0));
  if (i0 < iters) compute(st_of(i0), 0, xv[0], acc);
  __syncthreads();

  // Sums of the four waves, one m-tile at a time through the ring, added in
  // wave order; each wave finishes a quarter of the column tiles.
  f32x4* const red = reinterpret_cast<f32x4*>(&ring[0][0][0]);     // [kWaves][kStripTiles][64]
  static_assert(kWaves * kStripTiles * 64 * 16 <= kWaves * kRing * kSlot, "the cross-wave sum fits the ring");
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (i > 0) __syncthreads();
#pragma unroll
    for (int t = 0; t < kStripTiles; ++t) red[(wave * kStripTiles + t) * 64 + lane] = acc[t][i];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kStripTiles / kWaves; ++j) {
      const int t = wave * (kStripTiles / kWaves) + j;
      f32x4 v = red[t * 64 + lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        const f32x4 o = red[(w * kStripTiles + t) * 64 + lane];
        v[0] += o[0]; v[1] += o[1]; v[2] += o[2]; v[3] += o[3];
      }
      const int col = c0 + 16 * t + i16;
      if (col >= C) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * i + 4 * grp + r;
        if (row >= M) continue;
        if (part)
          part[(size_t)split * partial_slab(M, C) + (size_t)row * C + col] = v[r];
        else
          dx[(size_t)row * C + col] = f32_bf16(v[r]);
      }
    }
  }
}

}  // namespace

size_t linear_act_skinny_bytes(int64_t m, int64_t n, int64_t k) {
  const int splits = plan_layer((n + 31) / 32, k).splits;
  return splits <= 1 ? 0 : round_up((size_t)splits * partial_slab(m, n) * sizeof(float), kWorkspaceAlign);
}

hipError_t launch_linear_act_skinny(const uint16_t* x, const uint8_t* q, const float* s, uint16_t* y,
                                    const LayerEpilogue& ep, int64_t m, int64_t n, int64_t k, void* ws,
                                    size_t ws_bytes, hipStream_t stream) {
  const StreamPlan p = plan_layer((n + 31) / 32, k);
  if (p.splits > 1 && (ws == nullptr || ws_bytes < linear_act_skinny_bytes(m, n, k))) return hipErrorInvalidValue;
  float* const part = p.splits > 1 ? static_cast<float*>(ws) : nullptr;
  const dim3 grid((uint32_t)((n + 31) / 32), (uint32_t)p.splits), block(kWaves * 64);
  const int gk = (int)((k + kBlock - 1) / kBlock);
  with_path(m, (int64_t)grid.x * grid.y, false, [&](auto path) {
    using P = decltype(path);
    hipLaunchKernelGGL((linear_act_skinny_kernel<P>), grid, block, 0, stream, x, q, s, y, part, (int)m, (int)n,
                       (int)k, gk, p.ss_per_split * (kSuper / P::KW), ep);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_join_layer(part, y, p.splits, m, n, 0, ep, stream);
}

size_t glu_skinny_bytes(int64_t m, int64_t n, int64_t k) {
  const int splits = plan_layer((n + 15) / 16, k).splits;
  return splits <= 1 ? 0 : round_up((size_t)(2 * splits) * partial_slab(m, n) * sizeof(float), kWorkspaceAlign);
}

hipError_t launch_glu_skinny(const uint16_t* x, const uint8_t* qg, const float* sg, const uint8_t* qu,
                             const float* su, uint16_t* h, const LayerEpilogue& ep, int64_t m, int64_t n,
                             int64_t k, void* ws, size_t ws_bytes, hipStream_t stream) {
  const StreamPlan p = plan_layer((n + 15) / 16, k);
  if (p.splits > 1 && (ws == nullptr || ws_bytes < glu_skinny_bytes(m, n, k))) return hipErrorInvalidValue;
  float* const part = p.splits > 1 ? static_cast<float*>(ws) : nullptr;
  const dim3 grid((uint32_t)((n + 15) / 16), (uint32_t)p.splits), block(kWaves * 64);
  const int gk = (int)((k + kBlock - 1) / kBlock);
  with_path(m, (int64_t)grid.x * grid.y, true, [&](auto path) {
    using P = decltype(path);
    hipLaunchKernelGGL((glu_skinny_kernel<P>), grid, block, 0, stream, x, qg, sg, qu, su, h, part, (int)m, (int)n,
                       (int)k, gk, p.ss_per_split * (kSuper / P::KW), ep);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_join_glu(part, h, p.splits, m, n, 0, ep, stream);
}

size_t input_gradient_skinny_bytes(int64_t m, int64_t n, int64_t k, int products) {
  const GradientPlan p = plan_gradient_skinny(n, k, products);
  if (p.splits <= 1) return 0;
  return round_up((size_t)p.splits * partial_slab(m, k) * sizeof(float), kWorkspaceAlign);
}

hipError_t launch_input_gradient_skinny(const uint16_t* a, const uint8_t* q, const float* s,
                                        const uint16_t* a2, const uint8_t* q2, const float* s2, int64_t lda,
                                        uint16_t* dx, int64_t m, int64_t n, int64_t k, void* ws,
                                        size_t ws_bytes, hipStream_t stream) {
  const GradientPlan p = plan_gradient_skinny(n, k, a2 ? 2 : 1);
  float* part = nullptr;
  if (p.splits > 1) {
    if (ws == nullptr || ws_bytes < input_gradient_skinny_bytes(m, n, k, a2 ? 2 : 1)) return hipErrorInvalidValue;
    part = static_cast<float*>(ws);
  }
  const dim3 grid((uint32_t)(p.strips * p.splits)), block(kWaves * 64);
  const int gk = (int)((k + kBlock - 1) / kBlock);
  if (m <= 16)
    hipLaunchKernelGGL((input_gradient_skinny_kernel<1>), grid, block, 0, stream, a, q, s, a2, q2, s2, (int)lda,
                       dx, part, (int)m, (int)k, (int)n, gk, p.strips, p.steps1, p.steps, p.steps_per_split);
  else
    hipLaunchKernelGGL((input_gradient_skinny_kernel<2>), grid, block, 0, stream, a, q, s, a2, q2, s2, (int)lda,
                       dx, part, (int)m, (int)k, (int)n, gk, p.strips, p.steps1, p.steps, p.steps_per_split);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_join_layer(part, dx, p.splits, m, k, 0, LayerEpilogue{}, stream);
}

}  // namespace fp8bl
