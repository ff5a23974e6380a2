// The main loop of the large-M kernels (described in gemm_large.hip) with the
// forms built on it: the plain linear and gated pair of gemm_large.hip and the
// layer operators' kernels of gemm_layer.hip.
#pragma once

#include "fp8bl_act.h"
#include "fp8bl_device.h"
#include "fp8bl_internal.h"

namespace fp8bl {

namespace {

constexpr int kBK = 64;                     // K per step (of the plain kernels), and of an LDS row of X
constexpr int kBM = 256;                    // X rows per tile (the plain kernels' and the tallest)
constexpr int kBN = 256;                    // weight rows per tile
constexpr int kWaves = 4;
constexpr int kThreads = kWaves * 64;
constexpr uint32_t kOob = 0x80000000u;      // buffer offset past every valid range

static_assert(kBK == 64, "the X chunk permutation assumes 128-byte LDS rows");

// s_waitcnt immediates (gfx9 encoding: vmcnt[3:0] + vmcnt_hi[15:14],
// expcnt[6:4], lgkmcnt[11:8]). vm_wait(n): at most n vector-memory
// operations of this wave still outstanding, no wait on the others.
constexpr int vm_wait(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }
constexpr int kLgkmWait0 = 0xC07F;         // lgkmcnt(0) only

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  // dword 3 = 0x00020000: raw (untyped) buffer, 32-bit format, the gfx9
  // family layout; offsets at or past `bytes` read as zero. The size is made
  // wave-uniform so the descriptor lives in scalar registers.
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0,
                                           __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2* lds_i32x2_ptr_t;

// Cache policy of the finished tile's bf16 stores: non-temporal (bit 1 of
// the buffer instruction's cache field on gfx950). Nothing in the kernel
// reads them back, and streaming them past the caches keeps more of X and
// the codes, which other tiles re-read, in L2 and the MALL: 1-3% on
// 16384 x 12288 x 3072 and 16384 x 3072 x 3072 (same box, A/B, identical
// outputs). Split-K partials keep the default policy: the reduce reads them.
constexpr int kNonTemporal = 2;

// What a kernel computes with the loop above.
enum Form {
  kPlain,     // y = x W^T
  kLayer,     // y = act(x W^T + bias) + residual, z = x W^T + bias
  kGlu,       // h = act(x Wg^T) * (x Wu^T), g, u: the wave's two weight blocks are the
              // gate and the up rows of the same 32 output columns
  kGradient,  // y = x W + x2 W2 (x2 may be null): the reduction runs over the weight's rows
};

// What the forms besides kPlain read and write.
struct LargeArgs {
  LayerEpilogue ep;          // kLayer, kGlu
  const uint16_t* x2;        // kGradient: the second product's left operand
  int ldx;                   // kGradient: row stride of x and x2, elements (a multiple of 8)
  int steps1;                // kGradient: steps of one product
  int tile0;                 // first tile column of the launch (tiles_n counts from it); split
                             // partials hold the columns from it on
};

// (q, s) is the weight; for GATED and kGlu it is the gate weight and (q2, s2)
// the up weight, and y receives the product of the pair. For kGradient N is
// the weight's row length and K the number of its rows.
// MB: 32-row blocks of X per tile (8, 4 or 2), STAGES: ring length. Fewer rows
// make a step shorter, so that the codes of a weight stream through faster
// when there are not 256 rows to multiply. KS: 64-wide blocks of K per step. With 2 a code load
// reads 128 bytes of 8 weight rows instead of 64 of 16, which HBM streams
// faster (the codes of a row then lie 128 bytes apart in LDS, swizzled as X),
// and there are half the barriers. kGradient's loads stay 16 rows x 64 bytes:
// the four waves read 256 bytes of a row between them.
template <bool SPLIT, bool GATED, Form FORM, int ACT, int MB = 8, int STAGES = 3, int KS = 1>
__device__ __forceinline__
void gemm_large_body(const uint16_t* __restrict__ x, const uint8_t* __restrict__ q,
                     const float* __restrict__ s, const uint8_t* __restrict__ q2,
                     const float* __restrict__ s2, uint16_t* y,
                     float* __restrict__ part, int M, int N, int K, int gk,
                     int tiles_m, int tiles_n, int kt_per_split, int splits, int steps_per_unit,
                     const LargeArgs& la) {
  static_assert(!(SPLIT && GATED), "the SwiGLU needs whole sums: no K split");
  static_assert(!GATED || (FORM == kPlain && MB == 8), "GATED is a form of its own");
  static_assert(MB == 8 || MB == 4 || MB == 2, "row blocks go in pairs, a ring of eight fragments");
  constexpr int kStages = STAGES;
  constexpr int kTileM = 32 * MB;
  static_assert(KS == (MB == 2 ? 2 : 1), "the load slots of the steps built");
  constexpr int kStep = kBK * KS;                               // K per step
  constexpr int kXBlock = kTileM * kBK;                         // bf16 elements of a 64-wide block of X
  constexpr int kXElems = KS * kXBlock;                         // and of one stage's X tile
  constexpr int kXLoads = kXElems * 2 / 16 / kThreads;          // 16-byte X loads per lane per step
  constexpr int kWBytes = kBN * kStep;                          // bytes of one stage's codes
  constexpr int kWLoads = kWBytes / 16 / kThreads;              // 16-byte code loads per lane per step
  static_assert(kXLoads == MB * KS, "one wave's X loads cover a quarter of a stage's rows");
  static_assert(kWLoads == 4 * KS, "one wave's code loads cover its 64 rows of a stage");
  constexpr int kScales = FORM == kGlu ? 2 : 1;                 // scale words per wave and step
  constexpr int kSElems = kScales * kWaves * 64 * 4 / 2;        // their slots (256 B each)
  constexpr int kStageElems = kXElems + kWBytes / 2 + kSElems;  // stage size in bf16 elements (MB = 8: 49 KB)
  constexpr int kLoadsPerStep = kXLoads + kWLoads + kScales;
  static_assert((kStageElems * 2) % 256 == 0, "stages keep the LDS bank phase of their rows");
  static_assert(kStages * kStageElems * 2 <= 160 * 1024, "the ring fits the CU's LDS");
  __shared__ __attribute__((aligned(1024))) uint16_t xs[kStages * kStageElems];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Output columns of a tile, and the first row of this wave's weight rows
  // within the tile's rows of its weight.
  constexpr int kTileN = GATED || FORM == kGlu ? kBN / 2 : kBN;
  const int wrow = GATED ? 64 * (wave & 1) : FORM == kGlu ? 32 * wave : 64 * wave;
  const uint8_t* const wq = (GATED && wave >= 2) ? q2 : q;
  const float* const wsc = (GATED && wave >= 2) ? s2 : s;

  // ---- Work units: (tile, K split) pairs, dealt to the persistent
  // workgroups round-robin (unit blockIdx.x + i * gridDim.x). Consecutive
  // workgroups sit on consecutive XCDs; the renumbering gives each XCD a
  // contiguous run of units, walked in groups of 8 M-tiles, so the tiles
  // running at once on an XCD share X and W rows in its L2.
  const int ntiles = tiles_m * tiles_n;
  const int units = ntiles * splits;
  const int my_units = (units - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  const int nkt = FORM == kGradient && la.x2 ? 2 * la.steps1 : (K + kStep - 1) / kStep;
  const int ldx = FORM == kGradient ? la.ldx : K;    // row stride of X
  // Split partials are [M, PN] slabs of the launch's columns, pc0 .. N.
  const int pc0 = FORM == kPlain ? 0 : la.tile0 * kTileN;
  const int PN = N - pc0;
  struct Unit {
    int m0, n0, kt0, nreal, split;
  };
  auto unit_of = [&](int i) -> Unit {
    Unit U{0, 0, 0, 0, 0};              // past the last unit: no live step
    if (i >= my_units) return U;
    const int u = (int)blockIdx.x + i * (int)gridDim.x;
    // (units no multiple of 8: the forward forms give the first XCDs one unit
    // more, 1 - 5% faster, 333 x 4300 x 1168 18.8 -> 17.9 us; the gradient is
    // 5 - 8% slower with it below a round of tiles)
    const int even = (u & 7) * (units >> 3) + (u >> 3);
    const int r = FORM == kLayer || FORM == kGlu ? even + min(u & 7, units & 7) : (units & 7) == 0 ? even : u;
    U.split = r / ntiles;
    const int id = r - U.split * ntiles;
    constexpr int GM = 8;
    const int group = id / (GM * tiles_n);
    const int first_m = group * GM;
    const int gsize = min(tiles_m - first_m, GM);
    const int in_group = id - group * GM * tiles_n;
    U.m0 = (first_m + in_group % gsize) * kTileM;
    U.n0 = (in_group / gsize + (FORM == kPlain ? 0 : la.tile0)) * kTileN;
    U.kt0 = U.split * kt_per_split;
    U.nreal = min(kt_per_split, nkt - U.kt0);
    return U;
  };

  // ---- X staging: load i of wave w fills LDS rows 64w + 8i .. +8 of a
  // stage; lane l lands on row (l / 8) of those, physical chunk l % 8, and
  // fetches the logical chunk that the swizzle stores there: (l % 8) ^
  // ((4i + l/16) % 8), one of two chunks by the parity of i. The per-lane
  // offsets (row within the tile and chunk) are fixed for the whole kernel;
  // the tile goes in the descriptor and the step's K offset in the scalar
  // offset of the load. (The hardware checks only the per-lane part against
  // the descriptor's size, which is what guards the rows past M: the K
  // offset of a real chunk stays inside its row.)
  const int xc_even = (lane & 7) ^ (lane >> 4);
  const int xc_odd = (lane & 7) ^ (4 + (lane >> 4));
  uint32_t xvo[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
    xvo[i] = (uint32_t)((8 * MB * wave + 8 * i + (lane >> 3)) * ldx * 2 + ((i & 1) ? xc_odd : xc_even) * 16);
  // codes (KS = 1): load i of wave w fills the stage's code rows 64w + 16i .. +16
  // (64 bytes each, the step's K range) from its weight rows wrow + 16i ..;
  // lane l lands on row (l / 4), physical 16-byte chunk l % 4, holding the
  // logical chunk (l % 4) ^ (l / 16) (the row's (row / 4) % 4), so the
  // decoding reads below are conflict-free. A wave loads, and later reads,
  // only its own rows.
  // kGlu: rows 0..31 of a wave's 64 are gate rows, the others the up rows of
  // the same columns (the first and the second half of the loads).
  // KS = 2: eight rows of 128 bytes a load, chunks swizzled as X's.
  // kGradient: a wave's 64 code rows are the step's 64 weight rows, 64 bytes
  // (its output columns) of each. Chunk c of row r is stored at
  // c ^ (2 ((r / 4) % 2)): the transposing reads below take 32 bytes from
  // each of eight rows at once, which then lie in distinct banks.
  const int wc = FORM == kGradient ? (lane & 3) ^ (2 * ((lane >> 4) & 1)) : (lane & 3) ^ (lane >> 4);
  uint32_t wvo[kWLoads];
#pragma unroll
  for (int i = 0; i < kWLoads; ++i) {
    if constexpr (FORM == kGradient)
      wvo[i] = (uint32_t)((16 * i + (lane >> 2)) * N + 64 * wave + 16 * wc);
    else if constexpr (KS == 2)
      wvo[i] = (uint32_t)((wrow + 8 * (FORM == kGlu ? i & 3 : i) + (lane >> 3)) * K +
                          16 * ((i & 1) ? xc_odd : xc_even));
    else
      wvo[i] = (uint32_t)((wrow + 16 * (FORM == kGlu ? i & 1 : i) + (lane >> 2)) * K + 16 * wc);
  }
  const uint32_t srange = (uint32_t)((((FORM == kGradient ? K : N) + kBlock - 1) / kBlock) * gk * 4);
  const __amdgpu_buffer_rsrc_t srs = make_rsrc(wsc, srange);
  __amdgpu_buffer_rsrc_t srs2;
  if constexpr (FORM == kGlu || FORM == kGradient) srs2 = make_rsrc(s2 ? s2 : s, srange);

  // The unit whose steps are being loaded (STAGES - 1 steps ahead of the one
  // being computed, so near the end of a unit it is the next one).
  Unit LU = unit_of(0);
  __amdgpu_buffer_rsrc_t xrs, xrs2, wrs, wrs2;
  bool lwave_live;
  int lsrow;
  auto set_load_unit = [&](const Unit& U) {
    LU = U;
    const uint32_t xrange = (uint32_t)(U.nreal > 0 ? min(M - U.m0, kTileM) * ldx * 2 : 0);
    xrs = make_rsrc(x + (size_t)U.m0 * ldx, xrange);
    lwave_live = U.n0 + wrow < N;
    lsrow = lwave_live ? (U.n0 + wrow) / kBlock : 0;
    if constexpr (FORM == kGradient) {
      // (the codes' descriptor follows the step: issue_w)
      xrs2 = make_rsrc((la.x2 ? la.x2 : x) + (size_t)U.m0 * ldx, xrange);
    } else {
      const uint32_t wrange = (uint32_t)(U.nreal > 0 ? max(min(N - U.n0, kTileN), 0) * K : 0);
      wrs = make_rsrc(wq + (size_t)U.n0 * K, wrange);
      if constexpr (FORM == kGlu) wrs2 = make_rsrc(q2 + (size_t)U.n0 * K, wrange);
    }
  };
  set_load_unit(LU);

  // Stage loads. `sb` is the stage's first element in xs (wave-uniform).
  // X load i (of kXLoads) and code load i (of kWLoads) as above; each sends a
  // 1 KB wave-wide piece straight into LDS.
  // kGradient: step kt of the unit belongs to the first or the second
  // product; `kbase` counts within it.
  auto second = [&](int kt) -> bool { return FORM == kGradient && LU.kt0 + kt >= la.steps1; };
  auto base_of = [&](int kt) -> int {
    return (LU.kt0 + kt - (second(kt) ? la.steps1 : 0)) * kStep;
  };
  auto issue_x = [&](int sb, int kt, int i) {
    const int kbase = base_of(kt);
    // K left in this step (0 past the unit's range): a chunk is read iff it
    // starts below it
    const int klim = kt < LU.nreal ? K - kbase : 0;
    const int b = i / MB, ib = i % MB;              // 64-wide block, load within it
    const bool in = ((ib & 1) ? xc_odd : xc_even) * 8 + kBK * b < klim;
    lds_ptr_t to = (lds_ptr_t)&xs[sb + b * kXBlock + (8 * MB * wave + 8 * ib) * kBK];
    const uint32_t koff = (uint32_t)((kbase + kBK * b) * 2);
    if (FORM == kGradient && second(kt))
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xrs2, to, 16, in ? xvo[ib] : kOob, koff, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xrs, to, 16, in ? xvo[ib] : kOob, koff, 0, 0);
  };
  auto issue_w = [&](int sb, int kt, int i) {
    const int kbase = base_of(kt);
    const int klim = kt < LU.nreal ? K - kbase : 0;
    // (a load fills 1 KB: 16 rows of 64 bytes or 8 of 128)
    lds_ptr_t to = (lds_ptr_t)&xs[sb + kXElems + (64 * wave * KS + 16 * i) * kBK / 2];
    if constexpr (FORM == kGradient) {
      // weight rows kbase.. (at most 64, fewer at the end), columns from the
      // tile's first: rows past the last lie past the range, columns past N
      // are pushed out of it
      const uint8_t* const base = (second(kt) ? q2 : q) + (size_t)kbase * N + LU.n0;
      const int rows = max(min(klim, kStep), 0);
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(base, (uint32_t)(rows > 0 ? rows * N - LU.n0 : 0));
      const bool in = LU.n0 + 64 * wave + 16 * wc < N;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to, 16, in ? wvo[i] : kOob, 0, 0, 0);
    } else {
      const bool kin = 16 * (KS == 2 ? ((i & 1) ? xc_odd : xc_even) : wc) < klim;
      if (FORM == kGlu && i >= 2 * KS)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(wrs2, to, 16, kin ? wvo[i] : kOob, (uint32_t)kbase, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(wrs, to, 16, kin ? wvo[i] : kOob, (uint32_t)kbase, 0, 0);
    }
  };
  // Weight scale: one per wave and step (the wave's 64 rows lie in one
  // 128-row scale block, the 64-wide step in one 128-wide block), moved into
  // the stage like the codes: every lane fetches the same word, so the
  // wave's 256-byte slot holds 64 copies. No load in the main loop writes a
  // register, so the only waits on global loads are the explicit ones below.
  // Waves past N and dead steps read zero. (The address is always formed,
  // block clamped, and pushed out of range when dead.)
  auto issue_s = [&](int sb, int kt) {
    const bool live = lwave_live & (kt < LU.nreal);
    lds_ptr_t to = (lds_ptr_t)&xs[sb + kXElems + kWBytes / 2 + wave * 128];
    if constexpr (FORM == kGradient) {
      // scale of (reduction block, the wave's output columns)
      const int rb = min(base_of(kt), K - 1) / kBlock;
      const uint32_t off = (uint32_t)((rb * gk + lsrow) * 4) + (live ? 0u : kOob);
      if (second(kt))
        __builtin_amdgcn_raw_ptr_buffer_load_lds(srs2, to, 4, off, 0, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(srs, to, 4, off, 0, 0, 0);
    } else {
      const int kb = min(((LU.kt0 + kt) * kStep) / kBlock, gk - 1);
      const uint32_t off = (uint32_t)((lsrow * gk + kb) * 4) + (live ? 0u : kOob);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(srs, to, 4, off, 0, 0, 0);
      if constexpr (FORM == kGlu)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            srs2, (lds_ptr_t)&xs[sb + kXElems + kWBytes / 2 + (kWaves + wave) * 128], 4, off, 0, 0, 0);
    }
  };
  auto issue_all = [&](int sb, int kt) {
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) issue_x(sb, kt, i);
#pragma unroll
    for (int i = 0; i < kWLoads; ++i) issue_w(sb, kt, i);
    issue_s(sb, kt);
  };
  auto read_s = [&](int sb, int i) -> float {
    return *reinterpret_cast<const float*>(&xs[sb + kXElems + kWBytes / 2 + (i * kWaves + wave) * 128]);
  };

  // Codes of weight block nb, K half j of a stage (the 16 codes of sub-steps
  // 2j and 2j+1): lane l reads row 64w + 32nb + l%32, logical chunk
  // l/32 + 2j, stored at chunk (l/32 + 2j) ^ ((l%32 / 4) % 4).
  // (KS = 2: rows of 128 bytes, chunk c of row r at c ^ ((r / 2) % 8).)
  const int crow = (64 * wave + (lane & 31)) * kStep;   // byte offset of the lane's row
  const int crd = crow + (((lane >> 5) ^ (((lane & 31) >> 1) & 7)) << 4);
  const int cswz = ((lane & 31) >> 2) & 3;
  const int crd0 = crow + ((((lane >> 5) + 0) ^ cswz) << 4);
  const int crd1 = crow + ((((lane >> 5) + 2) ^ cswz) << 4);
  // kGradient: the codes lie as [reduction row][output column]; a transposing
  // read gives a lane eight rows of one column. In each group of 16 lanes,
  // lanes 2r and 2r + 1 address the two halves of row r's 16 columns and lane
  // i receives column i, byte r from row r. The lane half takes the rows of
  // its X chunk (16h + 32(t/2) + 8(t%2) .. +8), its group of 16 lanes the
  // columns 16 ((l / 16) % 2) .. of the block.
  const int trow = (lane & 15) >> 1;
  const int tr0 = 64 * wave * kStep + (16 * (lane >> 5) + trow) * 64 + 8 * (lane & 1) + 16 * ((lane >> 4) & 1);
  const int trc[2] = {tr0 + 32 * (trow >> 2), tr0 + 32 * (1 ^ (trow >> 2))};
  auto read_w = [&](u32x4 (&c)[2], int sb, int j) {
    const uint8_t* const codes = reinterpret_cast<const uint8_t*>(&xs[sb + kXElems]);
    if constexpr (FORM == kGradient) {
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const i32x2 v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (lds_i32x2_ptr_t)(codes + trc[nb] + (32 * j + 8 * e) * 64));
          c[nb][2 * e] = (uint32_t)v[0];
          c[nb][2 * e + 1] = (uint32_t)v[1];
        }
    } else {
      const uint8_t* base = codes + (KS == 2 ? crd ^ (32 * j) : j ? crd1 : crd0);
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) c[nb] = *reinterpret_cast<const u32x4*>(base + nb * 32 * kStep);
    }
  };
  // X fragment f of a stage (sub-step t = f / MB, row block mb = f % MB): the
  // MFMA B operand of the 32 X rows 32mb.. and the 16 K of sub-step t.
  const int arow = lane & 31;
  const int ahalf = lane >> 5;
  const int aswz = (arow >> 1) & 7;
  auto read_xf = [&](int sb, int f) -> bf16x8 {
    const int t = f / MB, mb = f % MB;
    const int c = 2 * ahalf + 4 * ((t & 3) >> 1) + (t & 1);
    return *reinterpret_cast<const bf16x8*>(
        &xs[sb + (t >> 2) * kXBlock + arow * kBK + ((c ^ aswz) << 3) + mb * 32 * kBK]);
  };

  f32x16 acc[2][MB];
#pragma unroll
  for (int nb = 0; nb < 2; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[nb][mb][r] = 0.0f;

  // Workgroup barrier; the empty asm statements keep the compiler from
  // moving any memory access (LDS reads included) across it.
  auto wg_barrier = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // ---- Register pipeline of a step (kFrags fragments f = MB t + mb; sub-step
  // t runs the MFMAs of its MB X fragments against its two decoded weight
  // operands; the numbers below are those of MB = 8, 32 fragments a step):
  //  - X fragments are read four ahead of their MFMAs into a ring of eight;
  //    the last four of a step read the next stage, after the barrier;
  //  - sub-step t+1's weight operands are decoded during sub-step t (the
  //    next step's first ones during sub-step 3), codes read a K half ahead;
  //  - the loads of the step STAGES - 1 ahead are spread over fragments 0..24;
  //  - at fragment 24 the wave waits for its loads of the next step (the
  //    ones issued STAGES - 2 steps ago) and reads its codes and scale;
  //  - at fragment 28 the barrier: every wave is done with this stage (its
  //    last reads returned), and the next stage is complete.
  // fragments f..f+5 are live in the region of f, f+1; 8 slots keep the
  // slot of a fragment the same in every step
  constexpr int kRing = 8;
  constexpr int kAhead = 4;
  constexpr int kSubs = 4 * KS;           // sub-steps of 16 K
  constexpr int kFrags = kSubs * MB;
  static_assert(kFrags % kRing == 0, "a fragment's slot is the same in every step");
  // Fragment at which the next step's loads are waited for and its codes
  // read, and the one with the barrier, before the first read of the next
  // stage. Loads of the step STAGES - 1 ahead that are out by then.
  constexpr int kFragBar = kFrags - kAhead;
  constexpr int kFragWait = MB == 8 ? 24 : MB == 4 ? 8 : kFragBar;
  constexpr int kIssued = kXLoads + (MB == 4 ? 2 : kWLoads);
  constexpr int kInFlight = (kStages - 3) * kLoadsPerStep + kIssued;
  static_assert(kInFlight <= 63 && (kStages - 2) * kLoadsPerStep <= 63, "vmcnt holds the loads in flight");
  bf16x8 xr[kRing];
  u32x4 wdh[2][2];          // decoded weight operands (bf16 pairs), by sub-step parity
  u32x4 cA[2], cB[2];       // codes of K halves 0 and 1
  float sc[2], scn[2];      // this and the next step's scales of the two weight blocks (one unless kGlu)

  // Prologue: the first unit's first STAGES - 1 steps in flight (every unit has
  // at least that many, dead ones included); wait for step 0, then prepare its
  // first operands.
#pragma unroll
  for (int p = 0; p < kStages - 1; ++p) issue_all(p * kStageElems, p);
  __builtin_amdgcn_s_waitcnt(vm_wait((kStages - 2) * kLoadsPerStep));
  wg_barrier();
  read_w(cA, 0, 0);
  sc[0] = read_s(0, 0);
  sc[1] = kScales == 2 ? read_s(0, 1) : sc[0];
#pragma unroll
  for (int nb = 0; nb < 2; ++nb) wdh[0][nb] = __builtin_bit_cast(u32x4, dequant8(cA[nb][0], cA[nb][1], sc[nb]));
#pragma unroll
  for (int f = 0; f < kAhead; ++f) xr[f] = read_xf(0, f);

  const int col_lane = 64 * wave + 4 * ahalf;
  int S = 0;                 // stage of the step being computed
  int lkt = kStages - 2;     // step (of LU) most recently loaded
  for (int ci = 0; ci < my_units; ++ci) {
  for (int kt = 0; kt < steps_per_unit; ++kt) {
    // the step STAGES - 1 ahead: next step of LU, or step 0 of the next unit
    if (++lkt == steps_per_unit) {
      set_load_unit(unit_of(ci + 1));
      lkt = 0;
    }
    const int Sn = S == kStages - 1 ? 0 : S + 1;
    const int L = S == 0 ? kStages - 1 : S - 1;
    const int sb = S * kStageElems, sbn = Sn * kStageElems, sbl = L * kStageElems;

#pragma unroll
    for (int t = 0; t < kSubs; ++t) {
      if ((t & 1) == 0 && t + 2 < kSubs) read_w(t & 2 ? cA : cB, sb, t / 2 + 1);
#pragma unroll
      for (int mb = 0; mb < MB; mb += 2) {
        // one region: the MFMAs of fragments f, f+1 with their share of the
        // other work, in a fixed order relative to the other regions
        const int f = MB * t + mb;
        if (f == kFragWait) {
          // this wave's loads of the next step (issued STAGES - 2 steps ago)
          // have landed, with the later ones still in flight: read its codes
          // of K half 0 and its scale
          __builtin_amdgcn_s_waitcnt(vm_wait(kInFlight));
          read_w(cA, sbn, 0);
          scn[0] = read_s(sbn, 0);
          scn[1] = kScales == 2 ? read_s(sbn, 1) : scn[0];
        }
        if (f == kFragBar) {
          // every wave is done with this stage (its last reads returned)
          // and has put its part of the next stage in place
          __builtin_amdgcn_s_waitcnt(kLgkmWait0);
          wg_barrier();
          __builtin_amdgcn_sched_barrier(0);
        }
        // read ahead (the last four from the next stage, after the barrier)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int fa = f + j + kAhead;
          xr[fa % kRing] = fa < kFrags ? read_xf(sb, fa) : read_xf(sbn, fa - kFrags);
        }
        // the loads of the step STAGES - 1 ahead, into the stage freed by the last barrier
        if constexpr (MB == 8) {
          if (f <= 14) issue_x(sbl, lkt, (f >> 1) + 0);
          if (f >= 16 && f <= 22) issue_w(sbl, lkt, (f - 16) >> 1);
          if (f == 24) issue_s(sbl, lkt);
        } else if constexpr (MB == 4) {
          if (f <= 2) { issue_x(sbl, lkt, f); issue_x(sbl, lkt, f + 1); }
          if (f >= 4 && f <= 10) issue_w(sbl, lkt, (f - 4) >> 1);
          if (f == 12) issue_s(sbl, lkt);
        } else {
          if (f <= 2) { issue_x(sbl, lkt, f); issue_x(sbl, lkt, f + 1); }
          if (f >= 4 && f <= 10) { issue_w(sbl, lkt, f - 4); issue_w(sbl, lkt, f - 3); }
          if (f == 12) issue_s(sbl, lkt);
        }
        // the next sub-step's weight operands, a quarter (one block's half
        // K of the sub-step: four codes to bf16) per region: sub-steps 1..3
        // from this step's codes, the next step's sub-step 0 from its codes
        // read at fragment 24, in the two regions after the barrier
        auto piece = [&](int q4) {
          const int nb = q4 >> 1, half = q4 & 1;
          const int tn = (t + 1) % kSubs;      // sub-step being prepared
          const u32x4 (&c)[2] = tn & 2 ? cB : cA;
          const u32x2 v = dequant4(c[nb][2 * (tn & 1) + half], tn == 0 ? scn[nb] : sc[nb]);
          wdh[tn & 1][nb][2 * half] = v[0];
          wdh[tn & 1][nb][2 * half + 1] = v[1];
        };
        if (t < kSubs - 1) {
          constexpr int kPieces = 8 / MB;
#pragma unroll
          for (int i = 0; i < kPieces; ++i) piece((mb >> 1) * kPieces + i);
        } else if (f >= kFragBar) {
          constexpr int kPieces = MB == 2 ? 4 : 2;
#pragma unroll
          for (int i = 0; i < kPieces; ++i) piece((f - (MB == 2 ? kFrags - 2 : kFragBar)) + i);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
            acc[nb][mb + j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                __builtin_bit_cast(bf16x8, wdh[t & 1][nb]), xr[(f + j) % kRing], acc[nb][mb + j], 0, 0, 0);
        if constexpr (MB == 8) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
          __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }

    sc[0] = scn[0];
    sc[1] = scn[1];
    S = Sn;
  }

    // ---- Epilogue of unit ci (the next unit's first loads are already in
    // flight). acc[nb][mb][4g + e] is output row m0 + 32mb + l%32, column
    // n0 + 64w + 32nb + 8g + 4(l/32) + e. Stores go through a buffer
    // descriptor over the tile's valid rows, so rows past M are dropped by
    // the hardware; columns past N get an out-of-range offset. (The host
    // keeps 256 rows of the output within 2^31 bytes.)
    const Unit CU = unit_of(ci);
    const int rows = min(M - CU.m0, kTileM);
    const int col_base = CU.n0 + col_lane;
    if constexpr (GATED) {
      // Gate wave w < 2 finishes row blocks 0..3 of the slice and up wave
      // w + 2 row blocks 4..7; each sends its partner the other four, rounded
      // to bf16 (the SwiGLU rounds both products to bf16 first, so nothing
      // is lost). Two rounds of two row blocks go through the sender's own
      // 8 KB of X rows in the stage the last step used, 16 bytes per lane,
      // lane-contiguous; a barrier after the writes hands them over, one
      // after the partner's reads gives the rows back. Each finished row
      // block then leaves as whole 128-byte lines through the same rows, as
      // in the plain epilogue below. (Only N % 8 == 0 comes here.)
      const __amdgpu_buffer_rsrc_t yrs = make_rsrc(y + (size_t)CU.m0 * N, (uint32_t)(rows * N * 2));
      const int stage0 = (S == 0 ? 2 : S - 1) * kStageElems;
      int le;
      asm volatile("" : "=v"(le) : "0"(lane));
      uint8_t* const own = reinterpret_cast<uint8_t*>(&xs[stage0 + wave * 64 * kBK]);
      const uint8_t* const peer = reinterpret_cast<const uint8_t*>(&xs[stage0 + (wave ^ 2) * 64 * kBK]);
      const bool up = wave >= 2;
      const int er = le & 31, eh = le >> 5;
      const int rr = le >> 3;
      const int col8 = CU.n0 + wrow + 8 * (le & 7);
#pragma unroll
      for (int r2 = 0; r2 < 2; ++r2) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int nb = 0; nb < 2; ++nb) {
            const f32x16 a = up ? acc[nb][2 * r2 + i] : acc[nb][4 + 2 * r2 + i];
#pragma unroll
            for (int gp = 0; gp < 2; ++gp) {
              u32x4 v;
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = pack_bf16x2(a[8 * gp + 2 * e], a[8 * gp + 2 * e + 1]);
              *reinterpret_cast<u32x4*>(own + ((2 * i + nb) * 2 + gp) * 1024 + le * 16) = v;
            }
          }
        __builtin_amdgcn_s_waitcnt(kLgkmWait0);
        wg_barrier();
        u32x4 got[2][2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int gp = 0; gp < 2; ++gp)
              got[i][nb][gp] = *reinterpret_cast<const u32x4*>(peer + ((2 * i + nb) * 2 + gp) * 1024 + le * 16);
        __builtin_amdgcn_s_waitcnt(kLgkmWait0);
        wg_barrier();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint8_t* const buf = own + i * 4096;
#pragma unroll
          for (int nb = 0; nb < 2; ++nb) {
            const f32x16 a = up ? acc[nb][4 + 2 * r2 + i] : acc[nb][2 * r2 + i];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              u32x2 v;
#pragma unroll
              for (int w2 = 0; w2 < 2; ++w2) {
                const uint32_t mine = pack_bf16x2(a[4 * g + 2 * w2], a[4 * g + 2 * w2 + 1]);
                const uint32_t theirs = got[i][nb][g >> 1][2 * (g & 1) + w2];
                v[w2] = swiglu_bf16x2(up ? theirs : mine, up ? mine : theirs);
              }
              const int chunk = (4 * nb + g) ^ ((er >> 1) & 7);
              *reinterpret_cast<u32x2*>(buf + er * 128 + chunk * 16 + 8 * eh) = v;
            }
          }
          const int mb = (up ? 4 : 0) + 2 * r2 + i;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 8 * j + rr;
            const u32x4 v = *reinterpret_cast<const u32x4*>(buf + r * 128 + (((le & 7) ^ ((r >> 1) & 7)) * 16));
            const uint32_t off = col8 < N ? (uint32_t)(((32 * mb + r) * N + col8) * 2) : kOob;
            __builtin_amdgcn_raw_buffer_store_b128(v, yrs, off, 0, kNonTemporal);
          }
        }
      }
    } else if constexpr (FORM != kPlain && (!SPLIT || FORM == kGlu) || MB < 8) {
      // The forms' outputs go through LDS in fp32, kEpiRows rows of the wave's
      // 64 weight rows at a time: 256-byte rows, 16-byte chunk c of row r at
      // c ^ (r % 16), read back as four consecutive columns of a row per lane.
      // A lane keeps its columns' bias, and residual, z and y move as whole
      // 128-byte pieces of rows (kGlu: chunks 0..7 of a row are its 32 gate
      // columns, 8..15 the up columns, and a lane reads four of each). One
      // rounding per output. The LDS is the wave's own part of the stage the
      // last step used, X rows (8 KB) for MB = 8, else codes (4 or 8 KB): every
      // wave finished reading that stage before the last barrier, and only
      // this wave refills its part, with loads it issues after these reads
      // have returned.
      constexpr int kHalves = MB == 4 ? 2 : 1;
      constexpr int kEpiRows = 32 / kHalves;
      constexpr int kLanesRow = FORM == kGlu ? 8 : 16;        // lanes side by side on a row
      constexpr int kRowsRead = 64 / kLanesRow;
      const LayerEpilogue ep = FORM == kLayer || FORM == kGlu ? la.ep : LayerEpilogue{};
      int le;
      asm volatile("" : "=v"(le) : "0"(lane));
      const int er = le & 31, eh = le >> 5;
      const int cc = le % kLanesRow, rq = le / kLanesRow;
      const int col4 = CU.n0 + (FORM == kGlu ? 32 : 64) * wave + 4 * cc;
      const int last = (S == 0 ? kStages - 1 : S - 1) * kStageElems;
      uint8_t* const buf = reinterpret_cast<uint8_t*>(
          &xs[last + (MB == 8 ? wave * 64 * kBK : kXElems + wave * 64 * kStep / 2)]);
      // The lanes of one half write while the others wait: without the wave
      // barriers the compiler may run the two halves' lanes through the whole
      // epilogue one after the other, and reads would miss their writes.
      auto put = [&](int mb, int hf) {
        if constexpr (kHalves == 2) __builtin_amdgcn_wave_barrier();
        if (kHalves == 1 || (er >> 4) == hf) {
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const f32x16& a = acc[nb][mb];
              const u32x4 v = {__float_as_uint(a[4 * g]), __float_as_uint(a[4 * g + 1]),
                               __float_as_uint(a[4 * g + 2]), __float_as_uint(a[4 * g + 3])};
              const int c = 8 * nb + 2 * g + eh;
              *reinterpret_cast<u32x4*>(buf + (er & (kEpiRows - 1)) * 256 + ((c ^ (er & 15)) << 4)) = v;
            }
        }
        if constexpr (kHalves == 2) __builtin_amdgcn_wave_barrier();
      };
      auto get = [&](int r, int c) -> u32x4 {
        return *reinterpret_cast<const u32x4*>(buf + r * 256 + ((c ^ (r & 15)) << 4));
      };
      const bool quad = FORM == kGradient || (N & 3) == 0;    // (kGradient: a multiple of 16 always)
      if constexpr (SPLIT) {
        // fp32 partials: slab `split`, for kGlu slabs 2 split (gate) and 2 split + 1 (up)
        const size_t slab = partial_slab(M, PN);
        float* const p0 = part + (size_t)(FORM == kGlu ? 2 * CU.split : CU.split) * slab + (size_t)CU.m0 * PN;
        const uint32_t range = (uint32_t)(rows * PN * 4);
        const __amdgpu_buffer_rsrc_t prs = make_rsrc(p0, range);
        const __amdgpu_buffer_rsrc_t prs2 = make_rsrc(p0 + slab, FORM == kGlu ? range : 0);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int hf = 0; hf < kHalves; ++hf) {
            put(mb, hf);
#pragma unroll
            for (int j = 0; j < kEpiRows / kRowsRead; ++j) {
              const int r = kRowsRead * j + rq;
              const u32x4 v = get(r, cc);
              u32x4 v2 = {};
              if (FORM == kGlu) v2 = get(r, cc + 8);
              const uint32_t at = (uint32_t)(((32 * mb + kEpiRows * hf + r) * PN + col4 - pc0) * 4);
              if (quad) {
                const uint32_t off = col4 < N ? at : kOob;
                __builtin_amdgcn_raw_buffer_store_b128(v, prs, off, 0, 0);
                if (FORM == kGlu) __builtin_amdgcn_raw_buffer_store_b128(v2, prs2, off, 0, 0);
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t off = col4 + e < N ? at + 4 * e : kOob;
                  const uint32_t w = v[e], w2 = v2[e];
                  __builtin_amdgcn_raw_buffer_store_b32(w, prs, off, 0, 0);
                  if (FORM == kGlu) __builtin_amdgcn_raw_buffer_store_b32(w2, prs2, off, 0, 0);
                }
              }
            }
          }
      } else {
        const size_t tile = (size_t)CU.m0 * N;
        const uint32_t range = (uint32_t)(rows * N * 2);
        const __amdgpu_buffer_rsrc_t yrs = make_rsrc(y + tile, range);
        // (an absent array: no range, so nothing is read or written)
        const __amdgpu_buffer_rsrc_t rrs =
            make_rsrc(ep.residual ? ep.residual + tile : y + tile, ep.residual ? range : 0);
        const __amdgpu_buffer_rsrc_t brs = make_rsrc(ep.bias ? ep.bias : y, ep.bias ? (uint32_t)(N * 2) : 0);
        uint16_t* const save = FORM == kGlu ? ep.g : ep.z;
        const __amdgpu_buffer_rsrc_t zrs = make_rsrc(save ? save + tile : y + tile, save ? range : 0);
        const __amdgpu_buffer_rsrc_t urs = make_rsrc(ep.u ? ep.u + tile : y + tile, ep.u ? range : 0);
        float bias[4] = {};
        if (FORM == kLayer && ep.bias)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            bias[e] = bf16_f32(__builtin_amdgcn_raw_buffer_load_b16(brs, (uint32_t)((col4 + e) * 2), 0, 0));
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int hf = 0; hf < kHalves; ++hf) {
            put(mb, hf);
            const uint32_t at0 = (uint32_t)(((32 * mb + kEpiRows * hf + rq) * N + col4) * 2);
            const uint32_t step = (uint32_t)(2 * kRowsRead * N);
            if (quad) {
              const bool in = col4 < N;
              u32x2 res[kEpiRows / kRowsRead] = {};
              if (FORM == kLayer && ep.residual)
#pragma unroll
                for (int j = 0; j < kEpiRows / kRowsRead; ++j)
                  res[j] = __builtin_bit_cast(
                      u32x2, __builtin_amdgcn_raw_buffer_load_b64(rrs, in ? at0 + (uint32_t)j * step : kOob, 0, 0));
#pragma unroll
              for (int j = 0; j < kEpiRows / kRowsRead; ++j) {
                const int r = kRowsRead * j + rq;
                const uint32_t off = in ? at0 + (uint32_t)j * step : kOob;
                const u32x4 v = get(r, cc);
                float t[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] = __uint_as_float(v[e]) + bias[e];
                const u32x2 zo = {pack_bf16x2(t[0], t[1]), pack_bf16x2(t[2], t[3])};
                if (FORM != kGradient && save) __builtin_amdgcn_raw_buffer_store_b64(zo, zrs, off, 0, kNonTemporal);
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] = act_f32<ACT>(t[e]);
                if constexpr (FORM == kGlu) {
                  const u32x4 v2 = get(r, cc + 8);
                  float u[4];
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    u[e] = __uint_as_float(v2[e]);
                    t[e] *= u[e];
                  }
                  const u32x2 uo = {pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3])};
                  if (save) __builtin_amdgcn_raw_buffer_store_b64(uo, urs, off, 0, kNonTemporal);
                }
                if (FORM == kLayer && ep.residual) {
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    t[e] += __uint_as_float((e & 1) ? res[j][e >> 1] & 0xFFFF0000u : res[j][e >> 1] << 16);
                }
                const u32x2 yo = {pack_bf16x2(t[0], t[1]), pack_bf16x2(t[2], t[3])};
                __builtin_amdgcn_raw_buffer_store_b64(yo, yrs, off, 0, kNonTemporal);
              }
            } else {
              // rows are only 2-byte aligned: one element at a time
#pragma unroll 1
              for (int j = 0; j < kEpiRows / kRowsRead; ++j) {
                const int r = kRowsRead * j + rq;
                const u32x4 v = get(r, cc);
                u32x4 v2 = {};
                if (FORM == kGlu) v2 = get(r, cc + 8);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t off = col4 + e < N ? at0 + (uint32_t)j * step + 2 * e : kOob;
                  const uint32_t w = v[e], w2 = v2[e];
                  const float z = __uint_as_float(w) + bias[e], u = __uint_as_float(w2);
                  float t = act_f32<ACT>(z);
                  if (FORM == kGlu) t *= u;
                  if (FORM == kLayer && ep.residual)
                    t += bf16_f32(__builtin_amdgcn_raw_buffer_load_b16(rrs, off, 0, 0));
                  if (save) {
                    __builtin_amdgcn_raw_buffer_store_b16(f32_bf16(z), zrs, off, 0, 0);
                    if (FORM == kGlu) __builtin_amdgcn_raw_buffer_store_b16(f32_bf16(u), urs, off, 0, 0);
                  }
                  __builtin_amdgcn_raw_buffer_store_b16(f32_bf16(t), yrs, off, 0, 0);
                }
              }
            }
          }
      }
    } else if constexpr (!SPLIT) {
      const __amdgpu_buffer_rsrc_t yrs = make_rsrc(y + (size_t)CU.m0 * N, (uint32_t)(rows * N * 2));
      if ((N & 3) == 0) {
        if ((N & 7) == 0) {
          // Through LDS, so that every store writes whole 128-byte lines:
          // lane l holds four consecutive columns of row l % 32 of each
          // 32x32 block, so direct stores write 16 bytes into each of 32
          // rows, and eight of them fill a line; written to memory that way
          // a tile takes about three times as long. Each 32-row block of
          // this wave's 256 x 64 slice goes row-major into 4 KB of LDS (16-byte
          // chunk c of row r at chunk c ^ ((r / 2) % 8)), then comes back as
          // 16 bytes per lane, 8 lanes per 128-byte row, 8 rows per store.
          // The LDS is the wave's own 8 KB of X rows in the stage the last
          // step used: every wave finished reading that stage before the last
          // barrier, and only this wave refills those rows, with loads it
          // issues after these reads have returned.
          const int tb = (S == 0 ? 2 : S - 1) * kStageElems + wave * 64 * kBK;
          // (the lane index through an empty asm: the compiler would otherwise
          // compute every address below once, before the loops, and keep
          // them in registers the main loop needs)
          int le;
          asm volatile("" : "=v"(le) : "0"(lane));
          const int er = le & 31, eh = le >> 5;
          const int rr = le >> 3;                   // row within 8 for the read-back
          const int col8 = CU.n0 + 64 * wave + 8 * (le & 7);
#pragma unroll
          for (int mb = 0; mb < 8; ++mb) {
            uint16_t* buf = &xs[tb + (mb & 1) * 2048];
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const f32x16& a = acc[nb][mb];
                const u32x2 v = {pack_bf16x2(a[4 * g], a[4 * g + 1]), pack_bf16x2(a[4 * g + 2], a[4 * g + 3])};
                const int chunk = (4 * nb + g) ^ ((er >> 1) & 7);
                *reinterpret_cast<u32x2*>(reinterpret_cast<uint8_t*>(buf) + er * 128 + chunk * 16 + 8 * eh) = v;
              }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r = 8 * j + rr;
              const u32x4 v = *reinterpret_cast<const u32x4*>(
                  reinterpret_cast<const uint8_t*>(buf) + r * 128 + (((le & 7) ^ ((r >> 1) & 7)) * 16));
              const uint32_t off = col8 < N ? (uint32_t)(((32 * mb + r) * N + col8) * 2) : kOob;
              __builtin_amdgcn_raw_buffer_store_b128(v, yrs, off, 0, kNonTemporal);
            }
          }
        } else {
#pragma unroll
          for (int mb = 0; mb < 8; ++mb)
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const int col = col_base + 32 * nb + 8 * g;
                const uint32_t off = col < N ? (uint32_t)(((arow + 32 * mb) * N + col) * 2) : kOob;
                const f32x16& a = acc[nb][mb];
                const u32x2 v = {pack_bf16x2(a[4 * g], a[4 * g + 1]), pack_bf16x2(a[4 * g + 2], a[4 * g + 3])};
                __builtin_amdgcn_raw_buffer_store_b64(v, yrs, off, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
              }
        }
      } else {
#pragma unroll
        for (int mb = 0; mb < 8; ++mb)
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const int col = col_base + 32 * nb + 8 * (r >> 2) + (r & 3);
              const uint32_t off = col < N ? (uint32_t)(((arow + 32 * mb) * N + col) * 2) : kOob;
              __builtin_amdgcn_raw_buffer_store_b16(
                  __builtin_bit_cast(uint16_t, (__bf16)acc[nb][mb][r]), yrs, off, 0, 0);
              __builtin_amdgcn_sched_barrier(0);
            }
      }
    } else {
      const __amdgpu_buffer_rsrc_t prs =
          make_rsrc(part + (size_t)CU.split * partial_slab(M, PN) + (size_t)CU.m0 * PN,
                    (uint32_t)(rows * PN * 4));
      if (FORM == kGradient || (N & 3) == 0) {   // (kGradient: a multiple of 16 always)
        // fp32 partials through the same LDS slice, as whole lines: each
        // 32-row block of this wave's 256 x 64 slice row-major in its 8 KB
        // (256-byte rows, 16-byte chunk c of row r at c ^ (r % 16)), back as
        // 16 bytes per lane, 16 lanes per row, 4 rows per store.
        const int tb = (S == 0 ? 2 : S - 1) * kStageElems + wave * 64 * kBK;
        int le;
        asm volatile("" : "=v"(le) : "0"(lane));
        const int er = le & 31, eh = le >> 5;
        const int cc = le & 15, rq = le >> 4;
        const int col4 = CU.n0 + 64 * wave + 4 * cc;
        uint8_t* buf = reinterpret_cast<uint8_t*>(&xs[tb]);
#pragma unroll
        for (int mb = 0; mb < 8; ++mb) {
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const f32x16& a = acc[nb][mb];
              // (__builtin_bit_cast of a vector element read element 0 here:
              // the values go through __float_as_uint instead.)
              const u32x4 v = {__float_as_uint(a[4 * g]), __float_as_uint(a[4 * g + 1]),
                               __float_as_uint(a[4 * g + 2]), __float_as_uint(a[4 * g + 3])};
              const int c = 8 * nb + 2 * g + eh;
              *reinterpret_cast<u32x4*>(buf + er * 256 + ((c ^ (er & 15)) << 4)) = v;
            }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int r = 4 * j + rq;
            const u32x4 v = *reinterpret_cast<const u32x4*>(buf + r * 256 + ((cc ^ (r & 15)) << 4));
            const uint32_t off = col4 < N ? (uint32_t)(((32 * mb + r) * PN + col4 - pc0) * 4) : kOob;
            __builtin_amdgcn_raw_buffer_store_b128(v, prs, off, 0, 0);
          }
        }
      } else {
#pragma unroll
        for (int mb = 0; mb < 8; ++mb)
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const int col = col_base + 32 * nb + 8 * (r >> 2) + (r & 3);
              const uint32_t off = col < N ? (uint32_t)(((arow + 32 * mb) * PN + col - pc0) * 4) : kOob;
              __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[nb][mb][r]), prs, off, 0, 0);
              __builtin_amdgcn_sched_barrier(0);
            }
      }
    }
#pragma unroll
    for (int nb = 0; nb < 2; ++nb)
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[nb][mb][r] = 0.0f;
  }
  // The loads issued for the unit after the last one target the ring;
  // drain them before exit.
  __builtin_amdgcn_s_waitcnt(vm_wait(0));
}

}  // namespace

}  // namespace fp8bl
