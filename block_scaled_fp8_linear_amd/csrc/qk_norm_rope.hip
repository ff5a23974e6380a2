// Norm and rotation of query and key heads, alone or with the keys and values
// going into the E4M3 cache in the same pass, and the store by itself.
//
// Norm and rotation: with r = 1 / sqrt(mean(x^2) + eps), the weight w and the
// turn's factors c, s of each element, and xo, wo the other member of its pair,
//   out = r (x (w c) + xo (wo s)),
// w c and wo s being the same for all heads of a token. One wave takes a token
// (or a part of its heads), works the token's cosines and sines out once, one
// pair a lane, and shares them through LDS; no wave waits for another. Bound by
// the heads' bytes, each read and written once: 16384 tokens of 80 heads of 128
// take 125 us (5.4 TB/s), 512 tokens of 72 heads 7.0 us (2.7 TB/s; the angles'
// fp64 and one wave's chain of loads, sums and stores), of which a launch of
// nothing is about 3. (Times of calls one after another over changing inputs; where
// choices are compared below, replays of one call in a graph.)
//
// Store: a workgroup takes a run of tokens. Where a later token of the call has
// the same slot, the earlier one is not stored: the workgroup compares its run
// with every later slot first, while its heads are on their way. 8192 tokens of
// 8 heads of 128 take 15.4 us (3.3 TB/s), of which the comparison is 2.4; the fused
// call for 16 tokens of 64 and 8 heads 5.2 us on the GPU. Its keys are normed, turned
// and divided in fp64: in fp32 one code in 200000 was its neighbour's, where the value
// lies next to the border between them. That costs 8192 tokens of 64 and 8 heads 5%
// (75 us in all), 16 tokens nothing.
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

// fl32(x / s) for the codes. With y = fl32(1 / s), q0 = fl32(x y) and the residual
// r = x - q0 s (exact), fma(r, y, q0) is the quotient, but for its last bit where
// the quotient lies within 2^-22 of a last bit's step of the middle between two
// floats: of 2^14 pairs of bf16 mantissas none gets another code that way.
// Subnormal scales and their like, whose residuals are not exact, take the IEEE
// division.
__device__ __forceinline__ void quotients(float (&x)[8], float s) {
  if (s >= 0x1p-64f) {
    const float y = __fdiv_rn(1.0f, s);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float q0 = __fmul_rn(x[e], y);
      const float r = __builtin_fmaf(-q0, s, x[e]);
      x[e] = __builtin_copysignf(__builtin_fmaf(r, y, q0), x[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __fdiv_rn(x[e], s);
  }
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

// The heads [first, last) of q or k of one token, in steps of 64 / L, kAhead
// steps' loads on their way at a time (16384 tokens of 80 heads 138 us through the
// caches, 141 with one step, 138 with four).
constexpr int kAhead = 2;

template <int L, bool PAST>
struct Heads {
  const uint16_t* src;
  uint16_t* dst;
  const uint16_t* w;
  int64_t in_hs, out_hs;
  int first, last, sub;          // sub: the lane's head in a step
  bool mine;                     // the lane has elements
  u32x4 raw[kAhead];

  __device__ __forceinline__ void load(int h0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * (64 / L) + sub;
      raw[i] = mine && h < last ? get8<PAST>(src + h * in_hs) : u32x4{0, 0, 0, 0};
    }
  }
};

template <int L, bool PAST>
__device__ __forceinline__ Heads<L, PAST> heads_of(const HeadView& in, const HeadView& out, const uint16_t* w, int dim,
                                                   int token, int first, int last, int lane) {
  const int col = 8 * (lane % L);
  return Heads<L, PAST>{in.p + token * in.ts + col, out.p + token * out.ts + col, w + col, in.hs, out.hs, first, last,
                        lane / L, col < dim, {}};
}

// The first loads are on their way already.
template <int L, bool INTER, bool PAST>
__device__ __forceinline__ void rope_heads(Heads<L, PAST>& g, float inv_dim, double eps, const Chunk& ch,
                                           const float (&c)[8], const float (&s)[8]) {
  float a[8], b[8];
  {
    const u32x4 raw = g.mine ? *reinterpret_cast<const u32x4*>(g.w) : u32x4{0, 0, 0, 0};
    float own[8], other[8];
    unpack8(raw, own);
    unpack8(other_members<INTER>(raw, ch.partner), other);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = own[i] * c[i], b[i] = other[i] * s[i];
  }
  constexpr int G = 64 / L;
  for (int h0 = g.first; h0 < g.last; h0 += kAhead * G) {
    if (h0 != g.first) g.load(h0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (h0 + i * G >= g.last) break;
      const int h = h0 + i * G + g.sub;
      float x[8], o[8];
      unpack8(g.raw[i], x);
      unpack8(other_members<INTER>(g.raw[i], ch.partner), o);
      float sq = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = __builtin_fmaf(x[e], x[e], sq);
      float mean = head_sum<L>(sq) * inv_dim + (float)eps;
      if (__builtin_expect(!norm_in_range(mean), 0)) {
        const int by = norm_exponent<L>(x, eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = ldexpf(x[e], -by), o[e] = ldexpf(o[e], -by);
        mean = norm_scaled<L>(x, inv_dim, eps, by);
      }
      const float r = rsqrtf(mean);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = r * __builtin_fmaf(x[e], a[e], o[e] * b[e]);
      if (g.mine && h < g.last) put8<PAST>(g.dst + h * g.out_hs, pack8(x));
    }
  }
}

// One wave's part of a token's heads: steps of 64 / L heads, q's then k's. The
// first heads are loaded ahead of the angles.
template <int L, bool INTER, bool PAST>
__device__ __forceinline__ void rope_unit(const RopeArgs& g, int k_heads, int unit, int lane, float2* table) {
  const int token = unit / g.parts, part = unit % g.parts;
  constexpr int G = 64 / L;
  const int sq = (g.q.heads + G - 1) / G, sk = (k_heads + G - 1) / G;
  const int s0 = (sq + sk) * part / g.parts, s1 = (sq + sk) * (part + 1) / g.parts;
  auto q = heads_of<L, PAST>(g.q, g.qo, g.t.wq, g.t.dim, token, s0 * G, min(min(s1, sq) * G, g.q.heads), lane);
  auto k = heads_of<L, PAST>(g.k, g.ko, g.t.wk, g.t.dim, token, max(s0 - sq, 0) * G, min((s1 - sq) * G, k_heads), lane);
  if (s0 < sq) q.load(q.first);
  if (s0 >= sq) k.load(k.first);
  for (int p = lane; p < g.t.pairs; p += 64) table[p] = turn_of(g.t, g.t.axis[p], p, token);
  wave_sync();
  const Chunk ch = chunk_of<INTER>(lane, lane % L, g.t.pairs);
  float c[8], s[8];
  turn_factors<INTER>(table, ch, c, s);
  const float inv_dim = 1.0f / (float)g.t.dim;
  if (s0 < sq) rope_heads<L, INTER, PAST>(q, inv_dim, g.t.eps, ch, c, s);
  if (s1 > sq) {
    if (s0 < sq) k.load(k.first);
    rope_heads<L, INTER, PAST>(k, inv_dim, g.t.eps, ch, c, s);
  }
}

// The units of one wave. (tokens * parts is below 2^31: parts is above 1 only
// for few tokens.)
template <int L, bool INTER, bool PAST>
__device__ __forceinline__ void rope_waves(const RopeArgs& g, int k_heads, int block, int blocks, float2* table) {
  const int units = g.t.tokens * g.parts, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t u = (int64_t)block * kQkvWaves + wave; u < units; u += (int64_t)blocks * kQkvWaves)
    rope_unit<L, INTER, PAST>(g, k_heads, (int)u, threadIdx.x & 63, table);
}

template <int L, bool INTER, bool PAST>
__global__ __launch_bounds__(kQkvThreads)
void rope_kernel(RopeArgs g) {
  __shared__ float2 table[kQkvWaves][FP8BL_MAX_PAIRS];
  rope_waves<L, INTER, PAST>(g, g.k.heads, blockIdx.x, gridDim.x, table[threadIdx.x >> 6]);
}

constexpr int kMaxRun = 16;

// Bit r, in every lane: one of the slots that this wave looks at, behind token
// i0 + r, is that token's. The workgroup's threads look at four slots each a
// load, four loads on their way at a time (the first ahead of the run's own
// slots); slots outside the run's own range, as nearly all are where tokens lie in
// pages, need no more than that comparison (slots in random order take all: 16384
// tokens then take 44 us). Lane r of a wave holds the slot of token i0 + r.
__device__ __forceinline__ uint32_t later_ones(const int32_t* __restrict__ slots, int i0, int run, int run_slots,
                                               int tokens) {
  constexpr int kLoads = 4, kRound = kLoads * 4 * kQkvThreads;
  int v[kLoads][4];
  auto load = [&](int j0) {
#pragma unroll
    for (int f = 0; f < kLoads; ++f) {
      const int j = j0 + 4 * ((int)threadIdx.x + f * kQkvThreads);
      if (j + 4 <= tokens)
        __builtin_memcpy(v[f], slots + j, 16);
      else
#pragma unroll
        for (int e = 0; e < 4; ++e) v[f][e] = j + e < tokens ? slots[j + e] : -1;
    }
  };
  load(i0 + run);
  int lo = 0x7FFFFFFF, hi = -1;
  for (int r = 0; r < run; ++r) {
    const int s = __builtin_amdgcn_readlane(run_slots, r);
    lo = s >= 0 ? min(lo, s) : lo;
    hi = max(hi, s);
  }
  if (hi < 0) return 0;                      // padding alone
  const uint32_t span = (uint32_t)(hi - lo);
  bool again = false;                        // in the run itself: lane r looks at those behind its own
  for (int r = 1; r < run; ++r)
    again |= run_slots == __builtin_amdgcn_readlane(run_slots, r) && (int)(threadIdx.x & 63) < r;
  uint32_t found = 0;
  for (int j0 = i0 + run; j0 < tokens; j0 += kRound) {
    if (j0 != i0 + run) load(j0);
    bool near = false;
#pragma unroll
    for (int f = 0; f < kLoads; ++f)
#pragma unroll
      for (int e = 0; e < 4; ++e) near |= (uint32_t)v[f][e] - (uint32_t)lo <= span;
    if (near)
      for (int r = 0; r < run; ++r) {
        const int s = __builtin_amdgcn_readlane(run_slots, r);
#pragma unroll
        for (int f = 0; f < kLoads; ++f)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (s >= 0 && v[f][e] == s) found |= 1u << r;
      }
  }
  if (__any(found != 0)) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) found |= __shfl_xor(found, off, 64);
  }
  return found | (uint32_t)__ballot(again);
}

// The run's keys (normed and turned where FUSED) and values into the cache.
template <int L, bool INTER, bool FUSED>
__device__ __forceinline__ void store_run(const RopeArgs& g, const CacheArgs& k, int run_index) {
  __shared__ uint32_t found[kQkvWaves];
  __shared__ double2 tables[FUSED ? kMaxRun : 1][FUSED ? FP8BL_MAX_PAIRS : 1];
  constexpr int G = 64 / L, kBatch = 2;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i0 = run_index * k.run, run = min(k.run, g.t.tokens - i0);
  const int dim = g.t.dim, heads = g.k.heads;
  const int col = 8 * (lane % L);
  const bool mine = col < dim;
  const int steps = (heads + G - 1) / G;     // of a token's keys, and of its values
  const int items = run * 2 * steps;
  struct Item {
    int r, of_v, h;
  };
  auto item = [&](int u) { return Item{u / (2 * steps), u / steps % 2, u % steps * G + lane / L}; };
  u32x4 raw[kBatch];
  auto load = [&](int u0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int u = u0 + i * kQkvWaves;
      const Item t = item(u < items ? u : 0);
      const HeadView& in = t.of_v ? g.v : g.k;
      raw[i] = mine && u < items && t.h < heads
                   ? *reinterpret_cast<const u32x4*>(in.p + (i0 + t.r) * in.ts + t.h * in.hs + col)
                   : u32x4{0, 0, 0, 0};
    }
  };
  // lane r: the slot of token i0 + r
  const int run_slots = lane < run ? k.slots[i0 + lane] : -1;
  load(wave);              // on their way while the slots are compared

  const uint32_t mine_found = later_ones(k.slots, i0, run, run_slots, g.t.tokens);
  if (lane == 0) found[wave] = mine_found;
  if constexpr (FUSED)
    for (int p = tid; p < run * g.t.pairs; p += kQkvThreads)
      tables[p / g.t.pairs][p % g.t.pairs] =
          turn64<true>(g.t, g.t.axis[p % g.t.pairs], p % g.t.pairs, i0 + p / g.t.pairs);
  __syncthreads();
  uint32_t dead = found[0];
#pragma unroll
  for (int w = 1; w < kQkvWaves; ++w) dead |= found[w];
  dead = __builtin_amdgcn_readfirstlane(dead);

  const Chunk ch = chunk_of<INTER>(lane, lane % L, FUSED ? g.t.pairs : 8);
  float w[8], wo[8];
  if constexpr (FUSED) {
    const u32x4 wr = mine ? *reinterpret_cast<const u32x4*>(g.t.wk + col) : u32x4{0, 0, 0, 0};
    unpack8(wr, w);
    unpack8(other_members<INTER>(wr, ch.partner), wo);
  }
  for (int u0 = wave; u0 < items; u0 += kBatch * kQkvWaves) {
    if (u0 != wave) load(u0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int u = u0 + i * kQkvWaves;
      if (u >= items) break;
      const Item t = item(u);
      const int slot = __builtin_amdgcn_readlane(run_slots, t.r);
      if (slot < 0 || slot >= k.rows || (dead >> t.r & 1)) continue;
      float x[8], sc;
      unpack8(raw[i], x);
      if (FUSED && !t.of_v) {
        float o[8];
        double c[8], s[8], v[8], sq = 0.0, amax = 0.0;
        unpack8(other_members<INTER>(raw[i], ch.partner), o);
        turn_factors<INTER>(tables[t.r], ch, c, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fma((double)x[e], (double)x[e], sq);
        const double mean = head_sum<L>(sq) / dim + g.t.eps;
        const double n = mean == 0.0 ? 0.0 : 1.0 / sqrt(mean);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = n * fma((double)x[e] * (double)w[e], c[e], (double)o[e] * (double)wo[e] * s[e]);
          amax = fmax(amax, fabs(v[e]));
        }
        sc = (float)(head_max<L>(amax) / 448.0);
        if (sc == 0.0f) sc = 1.0f;
        const double inv = 1.0 / (double)sc;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (float)(v[e] * inv);
      } else {
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
        sc = __fdiv_rn(head_max<L>(amax), 448.0f);
        if (sc == 0.0f) sc = 1.0f;
        quotients(x, sc);
      }
      if (mine && t.h < heads) {
        const size_t row = (size_t)slot * heads + t.h;
        const u32x2 codes = {e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7])};
        *reinterpret_cast<u32x2*>((t.of_v ? k.vc : k.kc) + row * dim + col) = codes;
        if (col == 0) (t.of_v ? k.vs : k.ks)[row] = sc;
      }
    }
  }
}

template <int L>
__global__ __launch_bounds__(kQkvThreads)
void store_kernel(RopeArgs g, CacheArgs k) {
  store_run<L, false, false>(g, k, blockIdx.x);
}

// The first workgroups store, the others norm and turn q.
template <int L, bool INTER, bool PAST>
__global__ __launch_bounds__(kQkvThreads)
void rope_store_kernel(RopeArgs g, CacheArgs k, int runs) {
  __shared__ float2 table[kQkvWaves][FP8BL_MAX_PAIRS];
  if ((int)blockIdx.x < runs) {
    store_run<L, INTER, true>(g, k, blockIdx.x);
    return;
  }
  rope_waves<L, INTER, PAST>(g, 0, (int)blockIdx.x - runs, (int)gridDim.x - runs, table[threadIdx.x >> 6]);
}

// Waves to a token: as many as there are steps of 64 / L heads where few
// tokens would leave the chip empty, one where there are enough. Each works the
// angles out for itself, so more waves than fill the chip cost: 512 tokens of 72
// heads of 128 take 8.3 us with two waves, 7.3 with four, 7.5 with eight, 9.4 with 16;
// 1024 tokens of them 10.5 with four, 12.1 with eight; 2048 tokens of 18 heads of 80 7.2
// with two, 9.5 with four; three heads of 64 the same with any number.
int parts_of(int64_t tokens, int64_t steps) {
  int64_t parts = 4096 / tokens;
  if (parts > steps) parts = steps;
  return parts < 1 ? 1 : (int)parts;
}

int steps_of(int64_t heads, int lanes) { return (int)((heads + 64 / lanes - 1) / (64 / lanes)); }

// Tokens to a workgroup that stores: one where tokens are few; four, whose keys
// and values then take two batches of loads a wave at eight heads of 128; sixteen
// where the comparison of the slots, which grows with the square of the tokens over
// the run, would weigh. By the tokens alone, though a run's other work grows with its
// heads; in us, with runs of 1, 2, 4, 8, 16:
//   1 head of 64     1024 tokens  5.4  5.0  5.4  6.9 10.2     8192  17.7 13.2 10.9 11.0 12.5
//                   16384        35.2 23.9 18.2 16.6 17.5    65536     -  166 92.7 66.9 54.9
//   8 heads of 128   1024 tokens  5.9  6.1  6.8  9.8 15.9     8192  22.4 18.2 17.2 18.2 21.7
//                   16384        43.7 32.3 28.2 27.1 29.6    65536     -  225  155  120  105
//   32 heads of 128  2048 tokens 16.7 17.8 21.3 29.5 53.7     8192  47.2 44.4 44.3 49.9 66.4
//                   16384         106 92.1 89.6 92.2  117    65536     -  464  382  359  358
// (2048 tokens of 32 heads lose most by the rule, 21.7 for 16.7.)
int run_of(int64_t tokens) { return tokens <= 1024 ? 1 : tokens <= 16384 ? 4 : kMaxRun; }

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
  template <int L, bool INTER>
  hipError_t launch() {
    RopeArgs g = rope_args(a);
    g.parts = parts_of(a.tokens, steps_of(a.q_heads, L) + steps_of(a.k_heads, L));
    const dim3 grid(blocks_of(a.tokens, g.parts)), block(kQkvThreads);
    if (past_caches(a.tokens * (a.q_heads + a.k_heads) * a.head_dim * 4))
      hipLaunchKernelGGL((rope_kernel<L, INTER, true>), grid, block, 0, stream, g);
    else
      hipLaunchKernelGGL((rope_kernel<L, INTER, false>), grid, block, 0, stream, g);
    return hipGetLastError();
  }
  template <int L>
  hipError_t run() {
    return a.interleaved ? launch<L, true>() : launch<L, false>();
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
    hipLaunchKernelGGL((store_kernel<L>), dim3((uint32_t)((a.tokens + k.run - 1) / k.run)), dim3(kQkvThreads), 0,
                       stream, g, k);
    return hipGetLastError();
  }
};

struct RopeStore {
  const fp8bl_qkv& a;
  hipStream_t stream;
  template <int L, bool INTER>
  hipError_t launch() {
    RopeArgs g = rope_args(a);
    const CacheArgs k = cache_args(a);
    const int runs = a.k_heads > 0 ? (int)((a.tokens + k.run - 1) / k.run) : 0;
    g.parts = parts_of(a.tokens, steps_of(a.q_heads, L));
    const dim3 grid(runs + (a.q_heads > 0 ? blocks_of(a.tokens, g.parts) : 0)), block(kQkvThreads);
    if (past_caches(a.tokens * a.q_heads * a.head_dim * 4))
      hipLaunchKernelGGL((rope_store_kernel<L, INTER, true>), grid, block, 0, stream, g, k, runs);
    else
      hipLaunchKernelGGL((rope_store_kernel<L, INTER, false>), grid, block, 0, stream, g, k, runs);
    return hipGetLastError();
  }
  template <int L>
  hipError_t run() {
    return a.interleaved ? launch<L, true>() : launch<L, false>();
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
