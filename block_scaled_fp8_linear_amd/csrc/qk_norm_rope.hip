// Norm and rotation of query and key heads, alone or with the keys and values
// going into the E4M3 cache in the same pass, and the store by itself.
//
// Norm and rotation: with r = 1 / sqrt(mean(x^2) + eps), the weight w and the
// turn's factors c, s of each element, and xo, wo the other member of its pair,
//   out = r (x (w c) + xo (wo s)),
// w c and wo s being the same for all heads of a token. One wave takes a token
// (or a part of its heads), works the token's cosines and sines out once, one
// pair a lane, and shares them through LDS; no wave waits for another.
//
// Store: a workgroup takes a run of tokens. Where a later token of the call has
// the same slot, the earlier one is not stored: the workgroup compares its run
// with every later slot first.
#include "fp8bl_ops.h"
#include "qkv_device.h"

namespace fp8bl {

namespace {

// Four E4M3 codes; quotients up to 448 (1 + 2^-23) round to 448, larger ones
// (of a subnormal scale) are held there.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  auto top = [](float v) { return fminf(fmaxf(v, -448.0f), 448.0f); };
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(top(a), top(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(top(c), top(d), lo, true);
}

struct RopeArgs {
  HeadView q, k, v, qo, ko;
  TurnArgs t;
  int parts;        // waves to a token's heads
};

struct CacheArgs {
  const int32_t* slots;
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  int rows, run;    // cache rows; tokens to a workgroup
};

// The heads [first, last) in steps of 64 / L of one token.
template <int L, bool INTER>
__device__ __forceinline__ void rope_heads(const HeadView& in, const HeadView& out, const uint16_t* w, int dim,
                                           float eps, int token, int first, int last, int lane, const Chunk& ch,
                                           const float (&c)[8], const float (&s)[8]) {
  const int col = 8 * (lane % L);
  const bool mine = col < dim;
  float a[8], b[8];
  {
    const u32x4 raw = mine ? *reinterpret_cast<const u32x4*>(w + col) : u32x4{0, 0, 0, 0};
    float own[8], other[8];
    unpack8(raw, own);
    unpack8(other_members<INTER>(raw, ch.partner), other);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = own[i] * c[i], b[i] = other[i] * s[i];
  }
  const uint16_t* const src = in.p + token * in.ts + col;
  uint16_t* const dst = out.p + token * out.ts + col;
  const float inv_dim = 1.0f / (float)dim;
  for (int h = first + lane / L; h - lane / L < last; h += 64 / L) {
    const bool live = mine && h < last;
    const u32x4 raw = live ? *reinterpret_cast<const u32x4*>(src + h * in.hs) : u32x4{0, 0, 0, 0};
    float x[8], o[8];
    unpack8(raw, x);
    unpack8(other_members<INTER>(raw, ch.partner), o);
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = __builtin_fmaf(x[i], x[i], sq);
    const float r = rsqrtf(head_sum<L>(sq) * inv_dim + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = r * __builtin_fmaf(x[i], a[i], o[i] * b[i]);
    if (live) *reinterpret_cast<u32x4*>(dst + h * out.hs) = pack8(x);
  }
}

// One wave's part of a token's heads: steps of 64 / L heads, q's then k's.
template <int L, bool INTER>
__device__ __forceinline__ void rope_unit(const RopeArgs& g, int k_heads, int unit, int lane, float2* table) {
  const int token = unit / g.parts, part = unit % g.parts;
  for (int p = lane; p < g.t.pairs; p += 64) table[p] = turn_of(g.t, g.t.axis[p], p, token);
  wave_sync();
  const Chunk ch = chunk_of<INTER>(lane, lane % L, g.t.pairs);
  float c[8], s[8];
  turn_factors<INTER>(table, ch, c, s);
  constexpr int G = 64 / L;
  const int sq = (g.q.heads + G - 1) / G, sk = (k_heads + G - 1) / G;
  const int s0 = (sq + sk) * part / g.parts, s1 = (sq + sk) * (part + 1) / g.parts;
  if (s0 < sq)
    rope_heads<L, INTER>(g.q, g.qo, g.t.wq, g.t.dim, g.t.eps, token, s0 * G, min(min(s1, sq) * G, g.q.heads), lane, ch,
                         c, s);
  if (s1 > sq)
    rope_heads<L, INTER>(g.k, g.ko, g.t.wk, g.t.dim, g.t.eps, token, max(s0 - sq, 0) * G,
                         min((s1 - sq) * G, k_heads), lane, ch, c, s);
}

// The units of one wave. (tokens * parts is below 2^31: parts is above 1 only
// for few tokens.)
template <int L, bool INTER>
__device__ __forceinline__ void rope_waves(const RopeArgs& g, int k_heads, int block, int blocks, float2* table) {
  const int units = g.t.tokens * g.parts;
  for (int64_t u = (int64_t)block * kQkvWaves + (threadIdx.x >> 6); u < units; u += (int64_t)blocks * kQkvWaves)
    rope_unit<L, INTER>(g, k_heads, (int)u, threadIdx.x & 63, table);
}

template <int L, bool INTER>
__global__ __launch_bounds__(kQkvThreads)
void rope_kernel(RopeArgs g) {
  __shared__ float2 table[kQkvWaves][FP8BL_MAX_PAIRS];
  rope_waves<L, INTER>(g, g.k.heads, blockIdx.x, gridDim.x, table[threadIdx.x >> 6]);
}

constexpr int kMaxRun = 16;

// Bit r: a token behind i0 + r has its slot.
template <int R>
__device__ __forceinline__ uint32_t later_ones(const int32_t* slots, int i0, int tokens, const int* run_slots) {
  int mine[R];
#pragma unroll
  for (int r = 0; r < R; ++r) mine[r] = run_slots[r];
  uint32_t found = 0;
  for (int j = i0 + 1 + (int)threadIdx.x; j < tokens; j += kQkvThreads) {
    const int v = slots[j];
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (v == mine[r] && j > i0 + r) found |= 1u << r;
  }
  return found;
}

// The run's keys (normed and turned where FUSED) and values into the cache.
template <int L, bool INTER, bool FUSED>
__device__ __forceinline__ void store_run(const RopeArgs& g, const CacheArgs& k, int run_index) {
  __shared__ int run_slots[kMaxRun];
  __shared__ uint32_t dead;
  __shared__ float2 tables[FUSED ? kMaxRun : 1][FUSED ? FP8BL_MAX_PAIRS : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int i0 = run_index * k.run, run = min(k.run, g.t.tokens - i0);
  if (tid < kMaxRun) run_slots[tid] = tid < run ? k.slots[i0 + tid] : -1;
  if (tid == 0) dead = 0;
  __syncthreads();
  const uint32_t found = k.run == 1   ? later_ones<1>(k.slots, i0, g.t.tokens, run_slots)
                         : k.run == 4 ? later_ones<4>(k.slots, i0, g.t.tokens, run_slots)
                                      : later_ones<kMaxRun>(k.slots, i0, g.t.tokens, run_slots);
  if (found) atomicOr(&dead, found);
  if constexpr (FUSED)
    for (int p = tid; p < run * g.t.pairs; p += kQkvThreads)
      tables[p / g.t.pairs][p % g.t.pairs] = turn_of(g.t, g.t.axis[p % g.t.pairs], p % g.t.pairs, i0 + p / g.t.pairs);
  __syncthreads();

  constexpr int G = 64 / L;
  const int dim = g.t.dim, heads = g.k.heads;
  const int col = 8 * (lane % L);
  const bool mine = col < dim;
  const Chunk ch = chunk_of<INTER>(lane, lane % L, FUSED ? g.t.pairs : 8);
  float w[8], wo[8];
  if constexpr (FUSED) {
    const u32x4 raw = mine ? *reinterpret_cast<const u32x4*>(g.t.wk + col) : u32x4{0, 0, 0, 0};
    unpack8(raw, w);
    unpack8(other_members<INTER>(raw, ch.partner), wo);
  }
  const float inv_dim = 1.0f / (float)dim;
  const int steps = (heads + G - 1) / G;     // of a token's keys, and of its values
  for (int u = wave; u < run * 2 * steps; u += kQkvWaves) {
    const int r = u / (2 * steps), of_v = u / steps % 2, h = u % steps * G + lane / L;
    const int slot = run_slots[r];
    if (slot < 0 || slot >= k.rows || (dead >> r & 1)) continue;
    const HeadView& in = of_v ? g.v : g.k;
    const bool live = mine && h < heads;
    const u32x4 raw = live ? *reinterpret_cast<const u32x4*>(in.p + (i0 + r) * in.ts + h * in.hs + col)
                           : u32x4{0, 0, 0, 0};
    float x[8];
    unpack8(raw, x);
    if (FUSED && !of_v) {
      float o[8], c[8], s[8], sq = 0.0f;
      unpack8(other_members<INTER>(raw, ch.partner), o);
      turn_factors<INTER>(tables[r], ch, c, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = __builtin_fmaf(x[i], x[i], sq);
      const float n = rsqrtf(head_sum<L>(sq) * inv_dim + g.t.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = n * __builtin_fmaf(x[i], w[i] * c[i], o[i] * (wo[i] * s[i]));
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
    amax = head_max<L>(amax);
    float sc = __fdiv_rn(amax, 448.0f);
    if (sc == 0.0f) sc = 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], sc);
    if (live) {
      const size_t row = (size_t)slot * heads + h;
      const u32x2 codes = {e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7])};
      *reinterpret_cast<u32x2*>((of_v ? k.vc : k.kc) + row * dim + col) = codes;
      if (col == 0) (of_v ? k.vs : k.ks)[row] = sc;
    }
  }
}

template <int L>
__global__ __launch_bounds__(kQkvThreads)
void store_kernel(RopeArgs g, CacheArgs k) {
  store_run<L, false, false>(g, k, blockIdx.x);
}

// The first workgroups store, the others norm and turn q.
template <int L, bool INTER>
__global__ __launch_bounds__(kQkvThreads)
void rope_store_kernel(RopeArgs g, CacheArgs k, int runs) {
  __shared__ float2 table[kQkvWaves][FP8BL_MAX_PAIRS];
  if ((int)blockIdx.x < runs) {
    store_run<L, INTER, true>(g, k, blockIdx.x);
    return;
  }
  rope_waves<L, INTER>(g, 0, (int)blockIdx.x - runs, (int)gridDim.x - runs, table[threadIdx.x >> 6]);
}

// Waves to a token: as many as there are steps of 64 / L heads where few
// tokens would leave the chip empty, one where there are enough.
int parts_of(int64_t tokens, int64_t steps) {
  int64_t parts = 4096 / tokens;
  if (parts > steps) parts = steps;
  return parts < 1 ? 1 : (int)parts;
}

int steps_of(int64_t heads, int lanes) { return (int)((heads + 64 / lanes - 1) / (64 / lanes)); }

int run_of(int64_t tokens) { return tokens <= 2048 ? 1 : tokens <= 8192 ? 4 : kMaxRun; }

RopeArgs rope_args(const fp8bl_qkv& a) {
  return RopeArgs{head_view(a.q, a.q_heads), head_view(a.k, a.k_heads), head_view(a.v, a.k_heads),
                  head_view(a.q_out, a.q_heads), head_view(a.k_out, a.k_heads), turn_args(a), 1};
}

CacheArgs cache_args(const fp8bl_qkv& a) {
  return CacheArgs{a.slots, a.k_cache, a.v_cache, a.k_scale, a.v_scale, (int)a.cache_rows, run_of(a.tokens)};
}

// A launch has fewer than 2^32 threads: past 2^22 workgroups, waves take
// several units.
uint32_t blocks_of(int64_t tokens, int parts) {
  const int64_t blocks = (tokens * parts + kQkvWaves - 1) / kQkvWaves;
  return (uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks);
}

struct Rope {
  const fp8bl_qkv& a;
  hipStream_t stream;
  template <int L>
  hipError_t run() {
    RopeArgs g = rope_args(a);
    g.parts = parts_of(a.tokens, steps_of(a.q_heads, L) + steps_of(a.k_heads, L));
    const dim3 grid(blocks_of(a.tokens, g.parts)), block(kQkvThreads);
    if (a.interleaved)
      hipLaunchKernelGGL((rope_kernel<L, true>), grid, block, 0, stream, g);
    else
      hipLaunchKernelGGL((rope_kernel<L, false>), grid, block, 0, stream, g);
    return hipGetLastError();
  }
};

struct Store {
  const fp8bl_qkv& a;
  hipStream_t stream;
  template <int L>
  hipError_t run() {
    RopeArgs g{};
    g.k = head_view(a.k, a.k_heads);
    g.v = head_view(a.v, a.k_heads);
    g.t.tokens = (int)a.tokens;
    g.t.dim = (int)a.head_dim;
    const CacheArgs k = cache_args(a);
    const uint32_t runs = (uint32_t)((a.tokens + k.run - 1) / k.run);
    hipLaunchKernelGGL((store_kernel<L>), dim3(runs), dim3(kQkvThreads), 0, stream, g, k);
    return hipGetLastError();
  }
};

struct RopeStore {
  const fp8bl_qkv& a;
  hipStream_t stream;
  template <int L>
  hipError_t run() {
    RopeArgs g = rope_args(a);
    const CacheArgs k = cache_args(a);
    const int runs = a.k_heads > 0 ? (int)((a.tokens + k.run - 1) / k.run) : 0;
    g.parts = parts_of(a.tokens, steps_of(a.q_heads, L));
    const dim3 grid(runs + (a.q_heads > 0 ? blocks_of(a.tokens, g.parts) : 0)), block(kQkvThreads);
    if (a.interleaved)
      hipLaunchKernelGGL((rope_store_kernel<L, true>), grid, block, 0, stream, g, k, runs);
    else
      hipLaunchKernelGGL((rope_store_kernel<L, false>), grid, block, 0, stream, g, k, runs);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_qk_norm_rope(const fp8bl_qkv& a, hipStream_t stream) {
  return with_lanes(a.head_dim, Rope{a, stream});
}
hipError_t launch_kv_store(const fp8bl_qkv& a, hipStream_t stream) {
  return with_lanes(a.head_dim, Store{a, stream});
}
hipError_t launch_qk_norm_rope_store(const fp8bl_qkv& a, hipStream_t stream) {
  return with_lanes(a.head_dim, RopeStore{a, stream});
}

}  // namespace fp8bl
