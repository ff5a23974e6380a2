// 8-bit integer GEMM:
//   Y[m,n] = bf16( float(sum_k xq[m,k] wq[n,k]) * (xs[m] * ws[n]) + bias[n] )
// with the sum exact in int32, so that neither tiles nor K splits change a bit
// of the result.
//
// A workgroup of four waves, 2 x 2, each with a wave tile of 32 WM x 32 WN
// outputs in blocks of v_mfma_i32_32x32x32_i8. One step is 128 of K, four slices
// of 32: a wave reads WM + WN operands of a slice from LDS while the WM WN
// products of the one before it run. (With 4 x 4 blocks a wave, the LDS delivers
// 128 KB and takes in 64 KB a step of 2048 matrix cycles: three quarters of
// what it can do. Narrower wave tiles would be bound by it.)
//
// Stages of (TM + TN) x 128 bytes are filled by loads that write LDS themselves,
// S steps ahead. The last operands of a stage are read during the step's third
// slice, so one barrier a step, before the fourth, tells both that the next
// stage has landed and that this one can be refilled: half of its loads are issued
// in the fourth slice, half in the next step's first, one behind a product (all in
// the fourth take 8192 x 8192 x 8192 from 451 to 480 us, 2048 x 5120 x 5120 from 59
// to 66; thirds in three slices 473).
//
// LDS rows are 128 bytes with the 16-byte chunks permuted by
// (row & 7) ^ ((row >> 3) & 1): 16 consecutive rows of one chunk lie in 16
// different bank groups.
//
// v_mfma_i32_32x32x32_i8: lane l supplies 16 codes of row l % 32 at K half
// l / 32, A (the weight) and B (X) alike; it holds the sums of X row l % 32 and
// weight rows 8 g + 4 (l / 32) + i, g and i from 0 to 3.
//
// MI355X: 8192 x 8192 x 8192 433 to 451 us from one card to the next (2.44 to 2.54
// POP/s), 8192 x 12288 x 4096 348 to 365, 2048 x 5120 x 5120 57, 512 x 5120 x 5120
// 25, 333 x 4300 x 1168 9, the matrix cores busy 59% of the time in the second. The
// loads bound the first two: without them 387.
//
// Rows past M or N and K past the end read as zero: buffer descriptors that
// cover the valid rows, and offsets out of range for chunks behind K.
#include "fp8bl_device.h"
#include "fp8bl_ops.h"

namespace fp8bl {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kBK = 128;             // K of a step
constexpr int kSlices = kBK / 32;
constexpr int kThreads = 256;
constexpr uint32_t kOob = 0x80000000u;

constexpr int vm_wait(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }
constexpr int kLgkmWait0 = 0xC07F;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, __builtin_amdgcn_readfirstlane((int)bytes),
                                           0x00020000);
}

struct GemmArgs {
  const int8_t* xq;
  const float* xs;
  const int8_t* wq;
  const float* ws;
  const uint16_t* bias;
  uint16_t* y;
  int32_t* part;
  int M, N, K;
  int tiles_m, tiles_n, splits, steps_per_unit, steps;
};

template <int WM, int WN, int S>
struct Tile {
  static constexpr int kTM = 64 * WM, kTN = 64 * WN;
  static constexpr int kStage = (kTM + kTN) * kBK;
  static constexpr int kRows = 1024 / kBK;                        // of a load
  static constexpr int kXLoads = kTM / 4 / kRows, kWLoads = kTN / 4 / kRows;    // for each wave and step
  static constexpr int kLoads = kXLoads + kWLoads, kHalf = kLoads / 2;
  static constexpr int kVectors = (2 * kTN + kTM) * 4;            // of the epilogue
  static constexpr int kRowsOut = WN >= 2 ? 4 * 32 * 128 : 0;     // and its rows
  static constexpr int kLds = S * kStage + kVectors + kRowsOut;
  static_assert(kLds <= 160 * 1024, "the stages, the epilogue's vectors and its rows fit the LDS");
  static constexpr int kStores = 2 * WM * WN;                     // of a wave's sums as bf16 (the splits' own are twice as many)
  static_assert((S - 2) * kLoads + kStores <= 63 && (S - 1) * kLoads <= 63, "outstanding loads fit the counter");
};

template <int WM, int WN, int S, bool SPLIT>
__global__ __launch_bounds__(kThreads, 1)
void gemm_int8_kernel(GemmArgs g) {
  using T = Tile<WM, WN, S>;
  constexpr int kTM = T::kTM, kTN = T::kTN, kStage = T::kStage;
  // The stages and the epilogue's vectors in one array: with several, the
  // compiler tells their accesses apart and waits for every load into LDS
  // before the next read of it.
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::kLds];
  float* const ep_ws = reinterpret_cast<float*>(&lds[S * kStage]);
  float* const ep_bias = ep_ws + kTN;
  float* const ep_xs = ep_bias + kTN;
  uint8_t* const rows_out = &lds[S * kStage + T::kVectors + (T::kRowsOut / 4) * (threadIdx.x >> 6)];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int M = g.M, N = g.N, K = g.K;

  // ---- Units (tile, K split), dealt to the persistent workgroups round-robin;
  // each XCD gets a contiguous run, walked in groups of 4 M-tiles.
  const int ntiles = g.tiles_m * g.tiles_n;
  const int units = ntiles * g.splits;
  const int my_units = (units - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  struct Unit {
    int m0, n0, step0, nsteps, split;
  };
  auto unit_of = [&](int i) -> Unit {
    Unit U{0, 0, 0, 0, 0};              // past the last unit: nothing to load
    if (i >= my_units) return U;
    const int u = (int)blockIdx.x + i * (int)gridDim.x;
    const int r = (units & 7) == 0 ? (u & 7) * (units >> 3) + (u >> 3) : u;
    U.split = r / ntiles;
    const int id = r - U.split * ntiles;
    constexpr int GM = 4;
    const int group = id / (GM * g.tiles_n);
    const int first_m = group * GM;
    const int gsize = min(g.tiles_m - first_m, GM);
    const int in_group = id - group * GM * g.tiles_n;
    U.m0 = (first_m + in_group % gsize) * kTM;
    U.n0 = (in_group / gsize) * kTN;
    U.step0 = U.split * g.steps_per_unit;
    U.nsteps = min(g.steps_per_unit, g.steps - U.step0);
    return U;
  };

  // ---- Loads. Load j of wave w fills kRows rows from (TM / 4) w + kRows j on:
  // lane l lands on row l / kChunks of them at physical chunk l % kChunks and
  // fetches the logical chunk that lies there.
  constexpr int kChunks = kBK / 16;
  const int lrow = lane / kChunks;
  auto logical = [&](int j) { return (lane & 7) ^ (lane >> 3) ^ (j & 1); };
  uint32_t xvo[T::kXLoads], wvo[T::kWLoads];
#pragma unroll
  for (int j = 0; j < T::kXLoads; ++j)
    xvo[j] = (uint32_t)(((kTM / 4) * wave + T::kRows * j + lrow) * K + logical(j) * 16);
#pragma unroll
  for (int j = 0; j < T::kWLoads; ++j)
    wvo[j] = (uint32_t)(((kTN / 4) * wave + T::kRows * j + lrow) * K + logical(j) * 16);
  Unit LU;
  __amdgpu_buffer_rsrc_t xrs, wrs;
  auto set_load_unit = [&](const Unit& U) {
    LU = U;
    xrs = make_rsrc(g.xq + (size_t)U.m0 * K, (uint32_t)(U.nsteps > 0 ? min(M - U.m0, kTM) * K : 0));
    wrs = make_rsrc(g.wq + (size_t)U.n0 * K, (uint32_t)(U.nsteps > 0 ? min(N - U.n0, kTN) * K : 0));
  };
  // load i (of kLoads) of step `kt` of the load unit into the stage at `sb`; behind
  // the unit's last step everything is out of range, without a scalar offset that
  // would pass the descriptor's size too
  auto issue = [&](int sb, int kt, int i) {
    const int kbase = (LU.step0 + kt) * kBK;
    const int klim = kt < LU.nsteps ? K - kbase : 0;
    const bool of_x = i < T::kXLoads;
    const int j = of_x ? i : i - T::kXLoads;
    const bool in = logical(j) * 16 < klim;
    const uint32_t vo = of_x ? xvo[of_x ? j : 0] : wvo[of_x ? 0 : j];
    const int row = of_x ? (kTM / 4) * wave + T::kRows * j : kTM + (kTN / 4) * wave + T::kRows * j;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(of_x ? xrs : wrs, (lds_ptr_t)&lds[sb + row * kBK], 16, in ? vo : kOob,
                                             (uint32_t)(klim > 0 ? kbase : 0), 0, 0);
  };

  // ---- Operands of slice s of a stage.
  const int r32 = lane & 31, half = lane >> 5;
  const int swz = (r32 & 7) ^ ((r32 >> 3) & 1);
  const int xrow = (32 * WM * wm + r32) * kBK, wrow = (kTM + 32 * WN * wn + r32) * kBK;
  auto read_x = [&](int sb, int s, int b) -> i32x4 {
    return *reinterpret_cast<const i32x4*>(&lds[sb + xrow + 32 * b * kBK + (((2 * s + half) ^ swz) << 4)]);
  };
  auto read_w = [&](int sb, int s, int b) -> i32x4 {
    return *reinterpret_cast<const i32x4*>(&lds[sb + wrow + 32 * b * kBK + (((2 * s + half) ^ swz) << 4)]);
  };

  auto wg_barrier = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // Prologue: the first S steps, half of the last; wait for the first of them.
  set_load_unit(unit_of(0));
  int lci = 0, lkt = 0;                // the next step to load: of unit lci
  auto next_load = [&] {
    if (++lkt == g.steps_per_unit) {
      lkt = 0;
      set_load_unit(unit_of(++lci));
    }
  };
#pragma unroll
  for (int a = 0; a < S; ++a) {
#pragma unroll
    for (int i = 0; i < (a == S - 1 ? T::kHalf : T::kLoads); ++i) issue(a * kStage, lkt, i);
    if (a < S - 1) next_load();
  }
  __builtin_amdgcn_s_waitcnt(vm_wait((S - 2) * T::kLoads + T::kHalf));
  wg_barrier();

  i32x4 xf[2][WM], wf[2][WN];
#pragma unroll
  for (int b = 0; b < WM; ++b) xf[0][b] = read_x(0, 0, b);
#pragma unroll
  for (int b = 0; b < WN; ++b) wf[0][b] = read_w(0, 0, b);

  i32x16 acc[WN][WM];
#pragma unroll
  for (int n = 0; n < WN; ++n)
#pragma unroll
    for (int m = 0; m < WM; ++m) acc[n][m] = i32x16{};

  int stage = 0;
  bool stored = false;                 // the last unit's tile was whole
  for (int ci = 0; ci < my_units; ++ci) {
    const Unit CU = unit_of(ci);
    for (int kt = 0; kt < g.steps_per_unit; ++kt) {
      const int sb = stage * kStage;
      const int nstage = stage + 1 == S ? 0 : stage + 1;
      const int sbn = nstage * kStage;
      const int psb = (stage == 0 ? S - 1 : stage - 1) * kStage;
      const bool last = kt == g.steps_per_unit - 1;
      // the epilogue's vectors, one element a thread: on their way during the
      // unit's last step
      uint32_t e_ws = 0, e_xs = 0, e_bias = 0;
      if (!SPLIT && last) {
        e_ws = __builtin_amdgcn_raw_buffer_load_b32(make_rsrc(g.ws + CU.n0, (uint32_t)min(N - CU.n0, kTN) * 4), tid * 4, 0, 0);
        e_xs = __builtin_amdgcn_raw_buffer_load_b32(make_rsrc(g.xs + CU.m0, (uint32_t)min(M - CU.m0, kTM) * 4), tid * 4, 0, 0);
        if (g.bias)
          e_bias = __builtin_amdgcn_raw_buffer_load_b16(make_rsrc(g.bias + CU.n0, (uint32_t)min(N - CU.n0, kTN) * 2), tid * 2, 0, 0);
      }
#pragma unroll
      for (int s = 0; s < kSlices; ++s) {
        if (s == kSlices - 1) {
          // this wave's reads of the stage have returned and its loads of the
          // next stage have landed; behind the barrier so have all waves'
          __builtin_amdgcn_s_waitcnt(kLgkmWait0);
          // (In a unit's first step the last unit's stores are newer than the next
          // stage, with S above 2: where all of them were issued, those of a whole
          // tile, they may take until the second step.)
          if (kt == 0 && ci > 0) {
            if (S > 2 && stored)
              __builtin_amdgcn_s_waitcnt(vm_wait((S - 2) * T::kLoads + T::kStores));
            else
              __builtin_amdgcn_s_waitcnt(vm_wait(0));
          } else {
            __builtin_amdgcn_s_waitcnt(vm_wait((S - 2) * T::kLoads));
          }
          if (last) __builtin_amdgcn_s_waitcnt(vm_wait(0));      // the epilogue's vectors
          if (!SPLIT && last) {
            asm volatile("" : "+v"(e_bias));     // not looked at before the wait above
            if (tid < kTN) ep_ws[tid] = __uint_as_float(e_ws), ep_bias[tid] = __uint_as_float(e_bias << 16);
            if (tid < kTM) ep_xs[tid] = __uint_as_float(e_xs);
            __builtin_amdgcn_s_waitcnt(kLgkmWait0);
          }
          wg_barrier();
        }
        const int cur = s & 1, nxt = cur ^ 1;
        const int rb = s == kSlices - 1 ? sbn : sb;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < WN; ++b) wf[nxt][b] = read_w(rb, (s + 1) % kSlices, b);
#pragma unroll
        for (int b = 0; b < WM; ++b) xf[nxt][b] = read_x(rb, (s + 1) % kSlices, b);
        if (s == kSlices - 1) {
#pragma unroll
          for (int i = 0; i < T::kHalf; ++i) issue(sb, lkt, i);
        }
        if (s == 0) {                            // the other half, into the stage before
#pragma unroll
          for (int i = T::kHalf; i < T::kLoads; ++i) issue(psb, lkt, i);
        }
#pragma unroll
        for (int n = 0; n < WN; ++n)
#pragma unroll
          for (int m = 0; m < WM; ++m)
            acc[n][m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[cur][n], xf[cur][m], acc[n][m], 0, 0, 0);
        // reads behind the first products, loads behind the others
        constexpr int kProducts = WM * WN, kReads = WM + WN, kEvery = kReads > kProducts / 2 ? 2 * kReads / kProducts : 1;
        constexpr int kFirst = kReads / kEvery, kRest = kProducts > kFirst ? kProducts - kFirst : 1;
#pragma unroll
        for (int i = 0; i < kProducts; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                     // MFMA
          if (i < kFirst) __builtin_amdgcn_sched_group_barrier(0x100, kEvery, 0);                // DS read
          if ((s == kSlices - 1 || s == 0) && i >= kFirst)
            __builtin_amdgcn_sched_group_barrier(0x020, (T::kHalf + kRest - 1) / kRest, 0);      // VMEM
        }
        __builtin_amdgcn_sched_barrier(0);
        if (s == 0) next_load();
      }
      stage = nstage;
    }

    // ---- Epilogue of unit ci.
    // With 16 blocks the sums stay in accumulation registers and are read out one
    // at a time: left to itself the compiler copies all of them at once and
    // spills what the loop keeps (8192 x 12288 x 4096 3% slower). It knows
    // nothing of the wait between the last products and these reads, so that is
    // here, for every block.
    constexpr bool kReadOut = WM * WN >= 16;
    if constexpr (kReadOut) {
#pragma unroll
      for (int n = 0; n < WN; ++n)
#pragma unroll
        for (int m = 0; m < WM; ++m) asm volatile("s_nop 15\n\ts_nop 15" : "+a"(acc[n][m]));
    }
    auto sum = [&](int n, int m, int i) {
      int v;
      if constexpr (kReadOut)
        asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(acc[n][m][i]));
      else
        v = acc[n][m][i];
      return v;
    };
    int le;
    asm volatile("" : "=v"(le) : "0"(lane));     // keeps the addresses below out of the loop's registers
    const int er = le & 31, eh = le >> 5;
    const int row0 = 32 * WM * wm + er;          // in the tile
    const int rows = M - CU.m0;
    const int col0 = 32 * WN * wn;
    if constexpr (SPLIT) {
      int32_t* const p = g.part + (size_t)CU.split * partial_slab(M, N);
#pragma unroll
      for (int m = 0; m < WM; ++m) {
        const int row = row0 + 32 * m;
#pragma unroll
        for (int n = 0; n < WN; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int col = CU.n0 + col0 + 32 * n + 8 * q + 4 * eh;
            const i32x4 v = {sum(n, m, 4 * q), sum(n, m, 4 * q + 1), sum(n, m, 4 * q + 2), sum(n, m, 4 * q + 3)};
            int32_t* const to = p + ((size_t)CU.m0 + row) * N + col;
            if (row < rows && col + 4 <= N)
              __builtin_memcpy(to, &v, 16);
            else if (row < rows)
              for (int i = 0; i < 4; ++i)
                if (col + i < N) to[i] = v[i];
          }
      }
    } else {
      // Two blocks of columns at a time go through LDS, 32 rows of 128 bytes for each
      // wave, and leave eight lanes a row: whole lines where N is a multiple of 64, and
      // those past the caches (8192 x 12288 x 4096 with its quantizer 388 us, 410 with
      // stores of 32 bytes a row straight from the registers; 16384 x 5120 x 5120 377
      // and 384; 4000 x 4300 x 4096, whose lines are in parts, 98 and 94). Lines in
      // parts are slower past the caches: 8191 x 8191 x 4096 277 us and 259 through
      // them, 287 from the registers.
      constexpr int kWide = WN >= 2 ? 2 : 1;
      const bool lines = kWide == 2 && N % 64 == 0;
      auto put = [&](int row, int col, u32x4 out) {
        uint16_t* const to = g.y + ((size_t)CU.m0 + row) * N + col;
        if (lines && row < rows && col < N)
          __builtin_nontemporal_store(out, reinterpret_cast<u32x4*>(to));
        else if (row < rows && col + 8 <= N)
          __builtin_memcpy(to, &out, 16);
        else if (row < rows)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (col + i < N) to[i] = (uint16_t)(out[i >> 1] >> (16 * (i & 1)));
      };
#pragma unroll
      for (int n0 = 0; n0 < WN; n0 += kWide) {
        float w[kWide][4][4], b[kWide][4][4];
#pragma unroll
        for (int j = 0; j < kWide; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int at = col0 + 32 * (n0 + j) + 8 * q + 4 * eh;
            const f32x4 wv = *reinterpret_cast<const f32x4*>(&ep_ws[at]);
            const f32x4 bv = *reinterpret_cast<const f32x4*>(&ep_bias[at]);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[j][q][i] = wv[i], b[j][q][i] = bv[i];
          }
#pragma unroll
        for (int m = 0; m < WM; ++m) {
          const int row = row0 + 32 * m;
          const float x = ep_xs[row];
#pragma unroll
          for (int j = 0; j < kWide; ++j)
#pragma unroll
            for (int p = 0; p < 2; ++p) {        // column groups 2 p and 2 p + 1
              __builtin_amdgcn_sched_barrier(0);   // a few sums at a time in registers
              uint32_t d[2][2];
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  v[i] = (float)sum(n0 + j, m, 4 * (2 * p + q) + i) * (x * w[j][2 * p + q][i]);
                  if (g.bias) v[i] += b[j][2 * p + q][i];
                }
                d[q][0] = pack_bf16x2(v[0], v[1]);
                d[q][1] = pack_bf16x2(v[2], v[3]);
              }
              // halves of the wave trade groups: each lane then has 8 columns in a row
              u32x4 out;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const auto t = __builtin_amdgcn_permlane32_swap(d[0][i], d[1][i], false, false);
                out[i] = t[0];
                out[2 + i] = t[1];
              }
              if constexpr (kWide == 2)          // into the wave's 32 rows of 128 bytes
                *reinterpret_cast<u32x4*>(&rows_out[er * 128 + (((4 * j + 2 * p + eh) ^ (er & 7)) << 4)]) = out;
              else
                put(row, CU.n0 + col0 + 16 * p + 8 * eh, out);
            }
          if constexpr (kWide == 2)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 8 * i + (le >> 3);
              const u32x4 out = *reinterpret_cast<const u32x4*>(&rows_out[r * 128 + (((le & 7) ^ (r & 7)) << 4)]);
              put(32 * WM * wm + 32 * m + r, CU.n0 + col0 + 32 * n0 + 8 * (le & 7), out);
            }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < WN; ++n)
#pragma unroll
      for (int m = 0; m < WM; ++m) acc[n][m] = i32x16{};
    stored = M - CU.m0 >= kTM && N - CU.n0 >= kTN;     // (m0 + kTM can pass 2^31)
    if constexpr (!SPLIT) wg_barrier();          // the vectors have been read
  }
  __builtin_amdgcn_s_waitcnt(vm_wait(0));        // loads behind the last step still target the LDS
}

// Sum of the K splits' partials with the epilogue, four columns a thread. Rows
// of partials start at any multiple of four bytes.
__global__ __launch_bounds__(256)
void join_int8_kernel(const int32_t* __restrict__ part, const float* __restrict__ xs, const float* __restrict__ ws,
                      const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int splits, int M, int N) {
  const int64_t groups = (N + 3) / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / groups;
  const int col = (int)(i - row * groups) * 4;
  if (row >= M) return;
  const size_t slab = partial_slab(M, N), at = (size_t)row * N + col;
  const float x = xs[row];
  if (col + 4 <= N) {
    i32x4 t = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      i32x4 p;
      __builtin_memcpy(&p, part + s * slab + at, 16);
      t += p;
    }
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = (float)t[j] * (x * ws[col + j]);
      if (bias) v[j] += bf16_f32(bias[col + j]);
    }
    const u32x2 out = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    __builtin_memcpy(y + at, &out, 8);
    return;
  }
  for (int j = 0; col + j < N; ++j) {
    int t = 0;
    for (int s = 0; s < splits; ++s) t += part[s * slab + at + j];
    float v = (float)t * (x * ws[col + j]);
    if (bias) v += bf16_f32(bias[col + j]);
    y[at + j] = f32_bf16(v);
  }
}

template <int WM, int WN, int S>
hipError_t launch_tiles(GemmArgs g, hipStream_t stream) {
  constexpr int tm = Tile<WM, WN, S>::kTM;
  static_assert(tm == Tile<WM, WN, S>::kTN, "the plan counts square tiles");
  static_assert(kBK == kInt8StepK, "the plan counts this kernel's steps");
  const Int8Cut c = cut_int8(g.M, g.N, g.K, tm, g.splits);
  g.steps = (int)c.steps;
  g.steps_per_unit = (int)c.steps_per_unit;
  g.splits = (int)c.splits;
  g.tiles_m = (int)c.tiles_m;
  g.tiles_n = (int)c.tiles_n;
  const int64_t most = (int64_t)device_cus() * (160 * 1024 / Tile<WM, WN, S>::kLds);
  const dim3 grid((uint32_t)(c.units < most ? c.units : most));
  if (g.splits == 1)
    hipLaunchKernelGGL((gemm_int8_kernel<WM, WN, S, false>), grid, dim3(kThreads), 0, stream, g);
  else
    hipLaunchKernelGGL((gemm_int8_kernel<WM, WN, S, true>), grid, dim3(kThreads), 0, stream, g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.splits == 1) return e;
  return launch_int8_join(g.part, g.xs, g.ws, g.bias, g.y, g.splits, g.M, g.N, stream);
}

}  // namespace

hipError_t launch_int8_join(const int32_t* part, const float* xs, const float* ws, const uint16_t* bias, uint16_t* y,
                            int splits, int64_t m, int64_t n, hipStream_t stream) {
  const int64_t threads = m * ((n + 3) / 4);
  hipLaunchKernelGGL(join_int8_kernel, dim3((uint32_t)((threads + 255) / 256)), dim3(256), 0, stream, part, xs, ws,
                     bias, y, splits, (int)m, (int)n);
  return hipGetLastError();
}

size_t int8_gemm_bytes(int64_t m, int64_t n, int64_t k) {
  if (m <= kInt8SkinnyRows) return int8_skinny_bytes(m, n, k);
  const Int8Plan p = plan_int8(m, n, k);
  return p.splits <= 1 ? 0 : round_up((size_t)p.splits * partial_slab(m, n) * sizeof(int32_t), kWorkspaceAlign);
}

hipError_t launch_int8_gemm(const int8_t* xq, const float* xs, const int8_t* wq, const float* ws,
                            const uint16_t* bias, uint16_t* y, int64_t m, int64_t n, int64_t k, void* workspace,
                            hipStream_t stream) {
  if (m <= kInt8SkinnyRows) return launch_int8_skinny(xq, xs, wq, ws, bias, y, m, n, k, workspace, stream);
  const Int8Plan p = plan_int8(m, n, k);
  const GemmArgs g{xq, xs, wq, ws, bias, y, static_cast<int32_t*>(workspace), (int)m, (int)n, (int)k, 0, 0, p.splits,
                   0, 0};
  switch (p.tile) {
    case 0: return launch_tiles<4, 4, 2>(g, stream);
    case 1: return launch_tiles<2, 2, 4>(g, stream);
    default: return launch_tiles<1, 1, 4>(g, stream);
  }
}

}  // namespace fp8bl
