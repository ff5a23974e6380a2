// The skinny-M kernel's loop (described in gemm_skinny.hip) with the forms
// built on it.
#pragma once

#include "fp8bl_act.h"
#include "fp8bl_device.h"
#include "fp8bl_internal.h"

namespace fp8bl {

namespace {

constexpr int kSuper = 256;               // K per super-step (16 chunks of 16 codes per row)
constexpr unsigned kXcds = 8;              // XCDs of an MI355X; workgroups are dealt to them in turn
constexpr uint32_t kOob = 0x80000000u;    // buffer offset past every valid range

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  // dword 3 = 0x00020000: raw (untyped) buffer descriptor of the gfx9
  // family; offsets at or past `bytes` read as zero.
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ u32x4 buf_load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// The weight is read once: its loads carry the non-temporal cache policy
// (bit 1 of the buffer instruction's cache field on gfx950), which on MI355X
// streams an 8000 x 8192 weight 5-10% faster than default-policy loads.
constexpr int kNonTemporal = 2;

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// s_waitcnt immediate (gfx9 encoding: vmcnt[3:0] + vmcnt_hi[15:14],
// expcnt[6:4], lgkmcnt[11:8]): at most n vector-memory operations of this
// wave outstanding, no wait on the others.
constexpr int vm_wait(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }
constexpr int kLgkmWait0 = 0xC07F;         // lgkmcnt(0) only

// The codes go global -> LDS directly into a ring of D slots per wave, X
// into D register sets, and each super-step's X loads are issued ahead of
// its code loads. Loads return in issue order, so X, which comes from L2,
// does not wait behind the codes coming from HBM. On MI355X (8000 x 8192,
// rotated weight copies, same box) against the kernel this one replaced,
// which staged the codes through registers into LDS with one super-step in
// flight (outputs bit-identical with the same start order): 16.2 against
// 16.8 us at M = 16, 13.7 against 14.8 at M = 8, 13.0 against 13.7 at
// M = 1. Two slots (one
// super-step in flight behind the one computed) are fastest: three and four
// were 2-14% slower, so the bytes in flight per CU are not what holds the
// rate.
//
// Every super-step issues the same number of loads (steps past the range
// read zero through the buffer descriptors), so one wait for at most
// (D - 1) * kLoads outstanding loads covers the codes and X of the
// super-step about to be computed.
// Forms: the plain linear, the linear with its epilogue (kSkinnyLayer), and
// the gated pair (kSkinnyGlu): there the workgroup's two 16-row tiles are the
// gate (q, s) and the up (q2, s2) rows of the same 16 output columns, so both
// sums of an output meet in one lane. With K splits that form writes the gate
// partials to slabs 0, 2, .. and the up partials to slabs 1, 3, ..
//
// XLDS: X goes through LDS like the codes, whole 512-byte rows at a time, and
// comes back in the operand's layout. Loaded straight into the operand's
// registers, each 16 lanes touch 16 rows, and with 16 rows of X its loads take
// as long as the codes'. KW is the K of a super-step: 256, or 128 (128 bytes of
// eight rows a code load) to halve the slots that then hold X too
// (gemm_layer_skinny.hip has what the choices measured).
enum SkinnyForm { kSkinnyPlain, kSkinnyLayer, kSkinnyGlu };

template <int MT, int NT, int WAVES, int D, SkinnyForm FORM, bool XLDS = false, int KW = kSuper>
__device__ __forceinline__
void gemm_skinny_body(const uint16_t* __restrict__ x, const uint8_t* __restrict__ q,
                      const float* __restrict__ s, const uint8_t* __restrict__ q2,
                      const float* __restrict__ s2, uint16_t* y,
                      float* __restrict__ part, int M, int N, int K, int gk,
                      int ss_per_split, const LayerEpilogue& ep) {
  static_assert(FORM != kSkinnyGlu || NT == 2, "gate and up tiles");
  constexpr int kSlot = NT * 16 * KW;         // one super-step's codes of the wave's tiles
  constexpr int kTileLoads = KW / 64;             // code loads of a 16-row tile, and its 64-wide K blocks
  constexpr int kLoads = (NT + 2 * MT) * kTileLoads;         // code and X loads per super-step
  static_assert((D - 1) * kLoads <= 63, "outstanding loads fit the vmcnt counter");
  static_assert(NT == 1 || NT == 2, "one or two 16-row tiles per workgroup");
  static_assert(kBlock % (16 * NT) == 0, "a workgroup's rows share one scale row");
  constexpr int kXSlot = XLDS ? MT * 16 * KW * 2 : 0;   // one super-step's X rows, where they go through LDS
  __shared__ __attribute__((aligned(1024))) uint8_t ring[WAVES][D][kSlot + kXSlot];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int kCols = FORM == kSkinnyGlu ? 16 : 16 * NT;   // output columns of the workgroup
  const int n0 = blockIdx.x * kCols;
  const int nss = (K + KW - 1) / KW;
  const int ss0 = blockIdx.y * ss_per_split;
  const int ss1 = min(ss0 + ss_per_split, nss);
  // No lambda below captures an array whose size is a template parameter
  // (the ring, the accumulators, the load offsets): hipcc then leaves the
  // host launch stub undefined, without a diagnostic.
  uint8_t* const wring = &ring[wave][0][0];

  const __amdgpu_buffer_rsrc_t wrs =
      make_rsrc(q + (size_t)n0 * K, (uint32_t)(min(N - n0, kCols) * K));
  const __amdgpu_buffer_rsrc_t wrs2 =
      make_rsrc((FORM == kSkinnyGlu ? q2 : q) + (size_t)n0 * K, (uint32_t)(min(N - n0, kCols) * K));
  const __amdgpu_buffer_rsrc_t xrs = make_rsrc(x, (uint32_t)(M * K * 2));
  // The workgroup's rows lie in one 128-row scale block (16 * NT divides 128).
  const float* const srow = s + (size_t)(n0 / kBlock) * gk;
  const float* const srow2 = (FORM == kSkinnyGlu ? s2 : s) + (size_t)(n0 / kBlock) * gk;
  const bool live1 = FORM == kSkinnyGlu || n0 + 16 < N;    // tile 1 (NT = 2) has rows

  // Code loads: instruction r of tile j brings rows 4r..4r+3, 256 bytes
  // each; lane i lands at byte 16*i of the instruction's 1 KB of the slot
  // and fetches logical chunk (i & 15) ^ row.
  constexpr int kRowsLoad = 1024 / KW;            // rows of a load
  constexpr int kChunks = KW / 16;                // 16-byte chunks of a row
  const int lrow4 = lane / kChunks;
  const int lchk = lane % kChunks;
  // (the swizzle's key of a row: 16 rows of one chunk in 16 distinct chunks of 256 bytes)
  auto wkey = [](int row) { return KW == 256 ? row : (row >> 1) & 7; };
  uint32_t woff[4];       // (the first kTileLoads) tile 0's; tile j adds j * 16 rows
#pragma unroll
  for (int r = 0; r < kTileLoads; ++r) {
    const int row = kRowsLoad * r + lrow4;
    woff[r] = (uint32_t)(row * K + (lchk ^ wkey(row)) * 16);
  }
  const uint32_t tile_stride = (uint32_t)(16 * K);
  const int bn = lane & 15;
  const int bg = lane >> 4;
  const uint32_t xoff = (uint32_t)((bn * K + bg * 16) * 2);
  const uint32_t xtile_stride = (uint32_t)(16 * K * 2);

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int count = ss1 - ss0;
  // Every workgroup walks its K range from its own starting super-step, so
  // that at any moment the GPU reads many K offsets at once rather than all
  // rows at one offset (rows 8 KB apart then pile onto a few HBM channels:
  // 30% slower at 8000 x 8192). Workgroups are dealt to the 8 XCDs in turn,
  // so starting workgroup w at w / 8 gives the workgroups on each XCD every
  // start; w itself gave each XCD only four (4% slower at M = 16, 1% at
  // M = 1). The order is fixed per workgroup: results are run-to-run
  // identical.
  const int rot = count > 0 ? (int)((blockIdx.x / kXcds) % (unsigned)count) : 0;
  auto ss_of = [&](int i) {            // i-th super-step of the range, rotated
    if (i >= count) return ss1;        // past the end: loads read nothing
    const int r = i + rot;
    return ss0 + (r >= count ? r - count : r);
  };

  u32x4 xv[D][MT][kTileLoads][2];
  // XLDS: a load brings 1 KB of X rows of 2 KW bytes; 16-byte chunk c of row b
  // is stored at c ^ (b % 16), so the reads (one chunk of 16 rows at a time)
  // hit 16 distinct chunks of 256 bytes.
  constexpr int kXRow = 2 * KW, kXChunks = KW / 8;
  const int xr2 = lane / kXChunks, xp = lane % kXChunks;
  auto issue = [&](int ss, int slot, u32x4 (&xa)[MT][kTileLoads][2]) {
    const bool live = ss < ss1;
    const uint32_t kb = (uint32_t)(ss * KW);
    uint8_t* base = wring + slot * (kSlot + kXSlot);
    if constexpr (XLDS) {
#pragma unroll
      for (int r = 0; r < 2 * kTileLoads * MT; ++r) {
        const int row = (1024 / kXRow) * r + xr2, c = xp ^ (row & 15);
        const bool kin = live && (int)kb + c * 8 < K;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(xrs, (lds_ptr_t)(base + kSlot + r * 1024), 16,
                                                 kin ? (uint32_t)((row * K + (int)kb + c * 8) * 2) : kOob, 0, 0, 0);
      }
    } else
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < kTileLoads; ++h) {
        const bool kin = live && (int)kb + (bg + 4 * h) * 16 < K;
        const uint32_t o = xoff + i * xtile_stride + (kb + (uint32_t)(64 * h)) * 2;
        xa[i][h][0] = buf_load16(xrs, kin ? o : kOob);
        xa[i][h][1] = buf_load16(xrs, kin ? o + 16 : kOob);
      }
#pragma unroll
    for (int r = 0; r < kTileLoads; ++r) {
      const int row = kRowsLoad * r + lrow4;
      const bool kin = live && (int)kb + ((lchk ^ wkey(row)) * 16) < K;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (FORM == kSkinnyGlu && j == 1)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(wrs2, (lds_ptr_t)(base + j * 16 * KW + r * 1024), 16,
                                                   kin ? woff[r] + kb : kOob, 0, 0, kNonTemporal);
        else
          __builtin_amdgcn_raw_ptr_buffer_load_lds(wrs, (lds_ptr_t)(base + j * 16 * KW + r * 1024), 16,
                                                   kin ? woff[r] + j * tile_stride + kb : kOob, 0, 0, kNonTemporal);
    }
  };
  auto compute = [&](int ss, int slot, const u32x4 (&xa)[MT][kTileLoads][2], f32x4 (&ac)[MT][NT]) {
    // A super-step spans two 128-column scale blocks: logical chunks 0..7
    // (h = 0, 1) take the first, chunks 8..15 (h = 2, 3) the second. A K
    // tail never reads the second block's scale unless it exists.
    const int kb = KW / kBlock * ss;
    const float s0 = kb < gk ? srow[kb] : 0.0f;
    const float s1 = KW > kBlock && kb + 1 < gk ? srow[kb + 1] : 0.0f;
    float t0 = s0, t1 = s1;          // tile 1's
    if constexpr (FORM == kSkinnyGlu) {
      t0 = kb < gk ? srow2[kb] : 0.0f;
      t1 = KW > kBlock && kb + 1 < gk ? srow2[kb + 1] : 0.0f;
    }
    const uint8_t* base = wring + slot * (kSlot + kXSlot);
    u32x4 xl[MT][kTileLoads][2];
    if constexpr (XLDS) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < kTileLoads; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            xl[i][h][e] = *reinterpret_cast<const u32x4*>(base + kSlot + (16 * i + bn) * kXRow +
                                                          (((2 * (bg + 4 * h) + e) ^ bn) << 4));
    }
    const u32x4 (&xo)[MT][kTileLoads][2] = XLDS ? xl : xa;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const bool tl = j == 0 || live1;
      const uint8_t* slab = base + j * 16 * KW;
#pragma unroll
      for (int h = 0; h < kTileLoads; ++h) {
        const float sc = tl ? (h < 2 ? (j ? t0 : s0) : (j ? t1 : s1)) : 0.0f;
        const u32x4 c = *reinterpret_cast<const u32x4*>(slab + bn * KW + (((bg + 4 * h) ^ wkey(bn)) << 4));
        const bf16x8 b0 = dequant8(c[0], c[1], sc);
        const bf16x8 b1 = dequant8(c[2], c[3], sc);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          ac[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xo[i][h][0]), b0, ac[i][j], 0, 0, 0);
          ac[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xo[i][h][1]), b1, ac[i][j], 0, 0, 0);
        }
      }
    }
  };

  // Iteration i computes the wave's super-step ss_of(wave + i * WAVES) from
  // slot i % D, after issuing iteration i + D - 1's loads into the slot that
  // iteration i - 1 has finished reading. The main loop runs whole rounds of
  // D iterations with no branch inside, so the compiler sees which register
  // set each load wrote and adds no wait of its own beyond the one below;
  // the last iters % D iterations run after it. Every register load issued
  // in the main loop is used (by the next round or the tail), so none is
  // dropped and the fixed count holds.
  constexpr int kAhead = D - 1;
#pragma unroll
  for (int p = 0; p < kAhead; ++p) issue(ss_of(wave + p * WAVES), p, xv[p]);
  const int iters = count > wave ? (count - wave + WAVES - 1) / WAVES : 0;
  int i0 = 0;
  for (; i0 + D <= iters; i0 += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      const int nslot = (u + kAhead) % D;
      // Its last reads have returned: the loads write LDS on their own, and
      // the compiler orders a read before them, not its data.
      __builtin_amdgcn_s_waitcnt(kLgkmWait0);
      issue(ss_of(wave + (i0 + u + kAhead) * WAVES), nslot, xv[nslot]);
      __builtin_amdgcn_s_waitcnt(vm_wait(kAhead * kLoads));
      compute(ss_of(wave + (i0 + u) * WAVES), u, xv[u], acc);
    }
  }
  // The last iterations' super-steps are already in flight; they issue
  // nothing more and wait for everything. (A load issued here would have
  // no use, and the compiler drops unused register loads, which would
  // leave a fixed wait count short.)
#pragma unroll
  for (int u = 0; u < D - 1; ++u) {
    if (i0 + u < iters) {
      __builtin_amdgcn_s_waitcnt(vm_wait(0));
      compute(ss_of(wave + (i0 + u) * WAVES), u, xv[u], acc);
    }
  }
  // Loads past the range still write (zeros) into the ring: let them land
  // before the ring is reused for the cross-wave sum.
  __builtin_amdgcn_s_waitcnt(vm_wait(0));
  __syncthreads();

  f32x4* red = reinterpret_cast<f32x4*>(&ring[0][0][0]);   // [WAVES][MT * NT][64]
  static_assert(WAVES * MT * NT * 64 * 16 <= WAVES * D * (kSlot + kXSlot), "the cross-wave sum fits the ring");
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[(wave * MT * NT + i * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  auto total = [&](int p) -> f32x4 {
    f32x4 t = red[p * 64 + lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      const f32x4 o = red[(w * MT * NT + p) * 64 + lane];
      t[0] += o[0]; t[1] += o[1]; t[2] += o[2]; t[3] += o[3];
    }
    return t;
  };
  if constexpr (FORM == kSkinnyGlu) {
    // each of the first MT waves finishes one m-tile of both products
    if (wave >= MT) return;
    const f32x4 tg = total(wave * NT), tu = total(wave * NT + 1);
    const int col = n0 + (lane & 15);
    if (col >= N) return;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = wave * 16 + (lane >> 4) * 4 + r;
      if (row >= M) continue;
      const size_t at = (size_t)row * N + col;
      if (gridDim.y == 1) {
        if (ep.g) {
          ep.g[at] = f32_bf16(tg[r]);
          ep.u[at] = f32_bf16(tu[r]);
        }
        y[at] = f32_bf16(act_any(ep.act, tg[r]) * tu[r]);
      } else {
        float* const p = part + (size_t)(2 * blockIdx.y) * partial_slab(M, N) + at;
        p[0] = tg[r];
        p[partial_slab(M, N)] = tu[r];
      }
    }
    return;
  }
  // Each of the first MT*NT waves finishes one (m-tile, n-tile) pair.
  const int pair = wave;
  if (pair >= MT * NT) return;
  const int i = pair / NT, j = pair % NT;
  const f32x4 t = total(pair);
  const int col = n0 + j * 16 + (lane & 15);
  if (col >= N) return;
  const float bias = FORM == kSkinnyLayer && ep.bias ? bf16_f32(ep.bias[col]) : 0.0f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = i * 16 + (lane >> 4) * 4 + r;
    if (row >= M) continue;
    if (gridDim.y == 1 && FORM == kSkinnyLayer) {
      const size_t at = (size_t)row * N + col;
      const float z = t[r] + bias;
      if (ep.z) ep.z[at] = f32_bf16(z);
      float v = act_any(ep.act, z);
      if (ep.residual) v += bf16_f32(ep.residual[at]);
      y[at] = f32_bf16(v);
    } else if (gridDim.y == 1) {
      const __bf16 v = (__bf16)t[r];
      y[(size_t)row * N + col] = __builtin_bit_cast(uint16_t, v);
    } else {
      part[(size_t)blockIdx.y * partial_slab(M, N) + (size_t)row * N + col] = t[r];
    }
  }
}

constexpr int kWaves = 4;
constexpr int kRing = 2;   // ring slots per wave: one super-step in flight behind the one computed

}  // namespace

}  // namespace fp8bl
