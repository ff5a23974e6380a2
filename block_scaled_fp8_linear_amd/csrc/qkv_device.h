// What the kernels between the QKV projection and its cache share: the lanes
// of a head, sums over them, and the angles of a token.
//
// A head of D elements lies in L lanes, the power of two from D / 8 on: lane c
// of them holds elements 8 c .. 8 c + 7 (none from D / 8 on), so a wave reads
// 64 / L heads with one 16-byte load a lane.
#pragma once

#include "fp8bl_device.h"
#include "fp8bl_qkv.h"

namespace fp8bl {

namespace {

constexpr int kQkvWaves = 4;
constexpr int kQkvThreads = kQkvWaves * 64;
constexpr int64_t kMaxBlocks = (int64_t)1 << 22;   // workgroups of a launch

struct HeadView {
  uint16_t* p;
  int64_t ts, hs;
  int heads;
};

inline HeadView head_view(const fp8bl_heads& h, int64_t heads) {
  return HeadView{h.data, h.token_stride, h.head_stride, (int)heads};
}

struct TurnArgs {
  const uint16_t* wq;
  const uint16_t* wk;
  const int32_t* positions;
  const float* inv_freq;
  int tokens, dim, pairs;
  double eps;
  uint8_t axis[FP8BL_MAX_PAIRS];
};

inline TurnArgs turn_args(const fp8bl_qkv& a) {
  TurnArgs t{a.q_weight, a.k_weight, a.positions, a.inv_freq, (int)a.tokens, (int)a.head_dim, (int)a.pairs,
             a.eps, {}};
  for (int i = 0; i < (int)a.pairs; ++i) t.axis[i] = a.axis[i];
  return t;
}

// Whether a call goes past the caches: what it reads and writes is more than
// the 256 MB of the last-level cache, so nothing of it would be found there by the
// next kernel. In replays of a graph norm and rotation of 16384 tokens of 80 heads of
// 128 take 120 us so and 126 through the caches (185 and 188 with a copy of the results behind
// them), of 2048 tokens 18.5 and 20.5 (28.3 and 25.9); their backward pass at
// 16384 tokens 185 and 198 (312 and 326), at 1024 20.3 and 18.8 (31.7 and 29.0);
// rows of eight heads of 128 read back 142 and 159 at 131072 tokens (342 and 357),
// 7.7 and 6.1 at 4096 (17.3 and 13.4).
inline bool past_caches(int64_t bytes) { return bytes > (int64_t)256 << 20; }

// Eight elements, past the caches or through them.
template <bool PAST>
__device__ __forceinline__ u32x4 get8(const uint16_t* p) {
  if constexpr (PAST) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  return *reinterpret_cast<const u32x4*>(p);
}
template <bool PAST>
__device__ __forceinline__ void put8(uint16_t* p, u32x4 v) {
  if constexpr (PAST)
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
  else
    *reinterpret_cast<u32x4*>(p) = v;
}

inline int head_lanes(int64_t dim) {
  int l = 2;
  while (8 * l < dim) l *= 2;
  return l;
}

// Calls f.template run<L>() with the L of a head dimension.
template <typename F>
hipError_t with_lanes(int64_t dim, F&& f) {
  switch (head_lanes(dim)) {
    case 2: return f.template run<2>();
    case 4: return f.template run<4>();
    case 8: return f.template run<8>();
    case 16: return f.template run<16>();
    default: return f.template run<32>();
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  return __hiloint2double(__builtin_amdgcn_mov_dpp(__double2hiint(v), CTRL, 0xF, 0xF, true),
                          __builtin_amdgcn_mov_dpp(__double2loint(v), CTRL, 0xF, 0xF, true));
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kHalfMirror = 0x141, kRowRor8 = 0x128;

// Sum (maximum) over the L lanes of a head, the same bits in each of them.
template <int L, typename T, typename Op>
__device__ __forceinline__ T head_reduce(T v, Op op) {
  v = op(v, dpp<kQuadXor1>(v));
  if constexpr (L >= 4) v = op(v, dpp<kQuadXor2>(v));
  if constexpr (L >= 8) v = op(v, dpp<kHalfMirror>(v));
  if constexpr (L >= 16) v = op(v, dpp<kRowRor8>(v));
  if constexpr (L >= 32) v = op(v, __shfl_xor(v, 16, 64));
  return v;
}
template <int L, typename T>
__device__ __forceinline__ T head_sum(T v) {
  return head_reduce<L>(v, [](T a, T b) { return a + b; });
}
template <int L, typename T>
__device__ __forceinline__ T head_max(T v) {
  return head_reduce<L>(v, [](T a, T b) { return a > b ? a : b; });
}

// Whether fp32 holds what a head's norm is made of, by its mean(x^2) + eps. Below,
// squares may have been lost (all of them where |x| < 2^-75, and eps itself below
// 2^-149); above, squares may have overflowed.
__device__ __forceinline__ bool norm_in_range(float mean) { return mean >= 0x1p-32f && mean <= 0x1p64f; }

// Heads out of that range are normed as x 2^-e with eps 2^-2e, which gives the same
// norm: e brings the larger of max |x| and sqrt(eps) next to 1. 16384 tokens of 80
// heads of 128 take 124 us where all heads are scaled, 123 where none is; their
// backward pass 187 and 185. (In fp64 without a scale instead the kernels take 166
// registers for 112 to 120, 3 waves a SIMD for 4.)
template <int L>
__device__ __forceinline__ int norm_exponent(const float (&x)[8], double eps) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = head_max<L>(amax);
  const int ex = __builtin_amdgcn_frexp_expf(amax), ee = __builtin_amdgcn_frexp_exp(eps) >> 1;
  return eps == 0.0 || (amax != 0.0f && ex > ee) ? ex : ee;
}
// mean(x^2) + eps of a head that is scaled already; infinite, for a norm and gradients
// of zeros, for a head of zeros without an eps.
template <int L>
__device__ __forceinline__ float norm_scaled(const float (&x)[8], float inv_dim, double eps, int e) {
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sq = __builtin_fmaf(x[i], x[i], sq);
  const float mean = head_sum<L>(sq) * inv_dim + (float)ldexp(eps, -2 * e);
  return mean == 0.0f ? __builtin_inff() : mean;
}

__device__ __forceinline__ void unpack8(u32x4 a, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(a[i] << 16);
    v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

// cos and sin of pair p of a token. The angle position * inv_freq reaches 2^31
// radians and more, and is reduced in fp64 without losing any of it: the product's
// rounding error e comes back with the rest, and quarter turns go off it in two parts,
// pi / 2 = h + l but for 2^-109. theta - q h is a multiple of 2^-52 (or theta is below
// 1), so the first fma is exact. What is left, at most pi / 4, is off by 2^-53 for
// angles below 2^40; where q itself is off by more, far past 2^48, whole quarter turns
// are taken. It goes through the two power series: to a^11 and a^10 (off by 2e-10), so
// that both come out rounded once to fp32, or to a^13 and a^12 where they stay fp64 (off
// by 4e-13).
template <bool FP64>
__device__ __forceinline__ double2 turn64(const TurnArgs& t, int axis, int p, int token) {
  constexpr double h = 1.57079632679489655800, l = 6.12323399573676603587e-17;
  const double at = (double)t.positions[(size_t)axis * t.tokens + token], f = (double)t.inv_freq[p];
  const double theta = at * f, e = fma(at, f, -theta);
  constexpr double whole = 6755399441055744.0;       // 1.5 2^52: a sum with it has the nearest integer in its low bits
  const double sum = fma(at, f * 0.63661977236758134308, whole), quarters = sum - whole;
  double a = fma(-quarters, h, theta) + fma(-quarters, l, e);
  if (fabs(a) > 1.0) a = 0.0;
  const double z = a * a;
  const double s11 = FP64 ? fma(z, 1.0 / 6227020800, -1.0 / 39916800) : -1.0 / 39916800;
  const double c10 = FP64 ? fma(z, 1.0 / 479001600, -1.0 / 3628800) : -1.0 / 3628800;
  const double s = a * fma(z, fma(z, fma(z, fma(z, fma(z, s11, 1.0 / 362880), -1.0 / 5040), 1.0 / 120), -1.0 / 6), 1.0);
  const double c = fma(z, fma(z, fma(z, fma(z, fma(z, c10, 1.0 / 40320), -1.0 / 720), 1.0 / 24), -0.5), 1.0);
  const int q = __double2loint(sum) & 3;
  const double fs = q & 1 ? c : s, fc = q & 1 ? s : c;
  return double2{q == 1 || q == 2 ? -fc : fc, q >= 2 ? -fs : fs};
}
__device__ __forceinline__ float2 turn_of(const TurnArgs& t, int axis, int p, int token) {
  const double2 v = turn64<false>(t, axis, p, token);
  return float2{(float)v.x, (float)v.y};
}

// Where the lane's chunk c of a head stands: in the first or second members of
// the half layout's pairs, among the interleaved pairs, or behind them.
struct Chunk {
  int partner;    // lane with the other members (half layout), or the lane itself
  int pair;       // pair of the chunk's first element
  float sign;     // of the sine: -1 first members, 1 second, 0 not turned
};
template <bool INTER>
__device__ __forceinline__ Chunk chunk_of(int lane, int c, int pairs) {
  const int e = 8 * c;
  if constexpr (INTER) return Chunk{lane, e / 2, e < 2 * pairs ? 1.0f : 0.0f};
  if (e < pairs) return Chunk{lane + pairs / 8, e, -1.0f};
  if (e < 2 * pairs) return Chunk{lane - pairs / 8, e - pairs, 1.0f};
  return Chunk{lane, 0, 0.0f};
}

// What the lane's elements are multiplied with in a turn, from the token's
// table of cosines and sines: out_i = x_i c_i + (other member)_i s_i.
template <bool INTER, typename T2, typename T>
__device__ __forceinline__ void turn_factors(const T2* table, const Chunk& ch, T (&c)[8], T (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (ch.sign == 0.0f) {
      c[i] = 1;
      s[i] = 0;
    } else if constexpr (INTER) {
      const T2 t = table[ch.pair + i / 2];
      c[i] = t.x;
      s[i] = i & 1 ? t.y : -t.y;
    } else {
      const T2 t = table[ch.pair + i];
      c[i] = t.x;
      s[i] = ch.sign * t.y;
    }
  }
}

// The other members of the lane's elements.
template <bool INTER>
__device__ __forceinline__ u32x4 other_members(u32x4 x, int partner) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if constexpr (INTER)
      o[i] = (x[i] << 16) | (x[i] >> 16);
    else
      o[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(partner << 2, (int)x[i]);
  return o;
}

// LDS written by a wave for itself: its writes are done before its reads.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace

}  // namespace fp8bl
