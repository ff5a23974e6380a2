// 8-bit integer linear at up to 32 rows: bound by the bytes of the weight, which
// is streamed once. The sums are exact in int32, so the order in which K is
// walked, split and joined does not change a bit of the result.
//
// A workgroup owns 16 NT weight rows and one K range (normally all of K), cut
// into super-steps of KW that go round-robin to its waves. Codes are loaded 4
// rows x 256 bytes (8 x 128) an instruction, straight into the wave's LDS slots
// (16-byte chunks permuted by the row, so that the operands' reads, one chunk of
// 16 rows, lie in 16 different bank groups), and X likewise. A wave reads only
// what it loaded: no barrier until the waves' sums meet.
//
// FUSED: one row of bf16: every workgroup quantizes it for itself, into LDS,
// while its first codes are on their way. That takes the place of the quantizer's
// launch and of the X loads.
//
// v_mfma_i32_16x16x64_i8: lane l supplies 16 codes of row l % 16 at K chunk
// l / 16, A (X) and B (the weight) alike; it holds the sums of X rows
// 4 (l / 16) .. +3 and weight row l % 16.
#include "fp8bl_device.h"
#include "fp8bl_ops.h"
#include "int8_row.h"

namespace fp8bl {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kSlots = 2;                 // of a wave: one super-step on its way behind the one computed
constexpr unsigned kXcds = 8;
constexpr uint32_t kOob = 0x80000000u;
constexpr int kNonTemporal = 2;           // the weight is read once

constexpr int vm_wait(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }
constexpr int kLgkmWait0 = 0xC07F;

struct SkinnyArgs {
  const void* x;            // codes, or bf16 where FUSED
  const float* xs;
  const int8_t* wq;
  const float* ws;
  const uint16_t* bias;
  uint16_t* y;
  int32_t* part;
  int M, N, K, k_split;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// The row that a workgroup quantizes for itself stays in registers between the
// maximum and the codes. In LDS it is whole super-steps long, zero behind K; 16
// more zeros stand for the operand's rows that are not there.
constexpr int kFusedElems = kInt8FusedK, kFusedCodes = kFusedElems + 16;

template <int MT, int NT, int WAVES, int KW, bool FUSED>
__global__ __launch_bounds__(WAVES * 64)
void gemm_int8_skinny_kernel(SkinnyArgs a) {
  constexpr int kSlab = 16 * KW;                 // 16 rows of a super-step
  constexpr int kSlabLoads = KW / 64;            // loads of it
  constexpr int kSlabRows = 1024 / KW, kChunksRow = KW / 16;      // rows of a load, 16-byte chunks of a row
  constexpr int kSlot = (NT + (FUSED ? 0 : MT)) * kSlab;
  constexpr int kLoads = kSlot / 1024;
  constexpr int kRing = WAVES * kSlots * kSlot;
  static_assert((kSlots - 1) * kLoads <= 63, "outstanding loads fit the counter");
  static_assert(kRing <= 160 * 1024, "the slots fit the LDS");
  static_assert(!FUSED || MT == 1, "one row");
  constexpr int kThreads = WAVES * 64, kChunks = kFusedElems / (kThreads * 8);
  // one array: with several the compiler waits for the loads into LDS at each read
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kRing + (FUSED ? kFusedCodes + 128 : 0)];
  uint8_t* const codes = &lds[kRing];
  float* const scales = reinterpret_cast<float*>(&lds[kRing + (FUSED ? kFusedCodes : 0)]);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int M = a.M, N = a.N, K = a.K;
  const int n0 = blockIdx.x * 16 * NT;
  const int nss = (K + KW - 1) / KW;
  const int each = a.k_split / KW, ss0 = blockIdx.y * each, ss1 = min(ss0 + each, nss);
  uint8_t* const ring = &lds[wave * kSlots * kSlot];

  const __amdgpu_buffer_rsrc_t wrs = make_rsrc(a.wq + (size_t)n0 * K, (uint32_t)(min(N - n0, 16 * NT) * K));
  const __amdgpu_buffer_rsrc_t xrs = make_rsrc(a.x, (uint32_t)(FUSED ? 0 : M * K));

  // Load r of a slab brings kSlabRows rows from kSlabRows r on: lane l lands at
  // byte 16 l of its 1 KB, at chunk l % kChunksRow of its row, and fetches that
  // chunk ^ key(row): 16 rows of one chunk lie in 16 different chunks of 256 bytes.
  auto key = [](int row) { return KW == 256 ? row : (row >> 1) & 7; };
  auto chunk = [&](int r) { return (lane % kChunksRow) ^ key(kSlabRows * r + lane / kChunksRow); };
  uint32_t off[4];        // (the first kSlabLoads: a lambda that captures an array sized by a template
                          // parameter leaves the host stub undefined)
#pragma unroll
  for (int r = 0; r < kSlabLoads; ++r) off[r] = (uint32_t)((kSlabRows * r + lane / kChunksRow) * K + chunk(r) * 16);
  const int count = ss1 - ss0;
  // each workgroup starts at a super-step of its own: many K offsets are read at
  // any time, not all rows at one
  const int rot = count > 0 ? (int)((blockIdx.x / kXcds) % (unsigned)count) : 0;
  auto ss_of = [&](int i) {
    if (i >= count) return ss1;
    const int r = i + rot;
    return ss0 + (r >= count ? r - count : r);
  };
  auto issue = [&](int ss, int slot) {
    const uint32_t kb = (uint32_t)(ss * KW);
    const int klim = ss < ss1 ? K - (int)kb : 0;
    uint8_t* const base = ring + slot * kSlot;
#pragma unroll
    for (int r = 0; r < kSlabLoads; ++r) {
      const bool in = chunk(r) * 16 < klim;
      if constexpr (!FUSED)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(xrs, (lds_ptr_t)(base + (NT + i) * kSlab + r * 1024), 16,
                                                   in ? off[r] + (uint32_t)(16 * i * K) + kb : kOob, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(wrs, (lds_ptr_t)(base + j * kSlab + r * 1024), 16,
                                                 in ? off[r] + (uint32_t)(16 * j * K) + kb : kOob, 0, 0,
                                                 kNonTemporal);
    }
  };
  const int r16 = lane & 15, g = lane >> 4;
  const int xend = nss * KW;                               // FUSED: bytes of the row of codes
  i32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  auto compute = [&](int ss, int slot, i32x4 (&ac)[MT][NT]) {
    const uint8_t* const base = ring + slot * kSlot;
#pragma unroll
    for (int h = 0; h < kSlabLoads; ++h) {
      const int c = g + 4 * h, at = r16 * KW + ((c ^ key(r16)) << 4);
      i32x4 xv[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if constexpr (FUSED) {
          xv[i] = *reinterpret_cast<const i32x4*>(codes + (r16 == 0 ? ss * KW + 16 * c : xend));
        } else {
          xv[i] = *reinterpret_cast<const i32x4*>(base + (NT + i) * kSlab + at);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const i32x4 wv = *reinterpret_cast<const i32x4*>(base + j * kSlab + at);
#pragma unroll
        for (int i = 0; i < MT; ++i) ac[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(xv[i], wv, ac[i][j], 0, 0, 0);
      }
    }
  };

  // The wave's super-steps, one on its way behind the one computed.
  auto lds_barrier = [] {                  // of LDS accesses alone: the codes' loads stay on their way
    __builtin_amdgcn_s_waitcnt(kLgkmWait0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  const int iters = count > wave ? (count - wave + WAVES - 1) / WAVES : 0;
  if constexpr (FUSED) {
    // x ahead of the codes, which come from further away: loads return in order
    const uint16_t* const x = static_cast<const uint16_t*>(a.x);
    u32x4 raw[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = (tid + kThreads * i) * 8;
      raw[i] = c < K ? *reinterpret_cast<const u32x4*>(x + c) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int p = 0; p < kSlots; ++p) issue(ss_of(wave + p * WAVES), p);
    uint32_t top = 0;                       // of magnitudes, which order like integers
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max((raw[i][j] << 16) & 0x7FFFFFFFu, raw[i][j] & 0x7FFF0000u));
    float amax = __uint_as_float(top);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
    if (lane == 0) scales[1 + wave] = amax;
    lds_barrier();
    amax = scales[1];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) amax = fmaxf(amax, scales[1 + w]);
    const RowScale rs = int8_scale(amax);
    if (tid == 0) scales[0] = rs.s;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if (8 * kThreads * i >= xend) break;
      const int c = (tid + kThreads * i) * 8;    // zeros behind K, to the end of the last super-step
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(raw[i][j] << 16);
        v[2 * j + 1] = __uint_as_float(raw[i][j] & 0xFFFF0000u);
      }
      const u32x2 q = codes8(v, rs);
      if (c < xend) *reinterpret_cast<u32x2*>(codes + c) = q;
    }
    if (tid < 2) *reinterpret_cast<u32x2*>(codes + xend + 8 * tid) = u32x2{0, 0};
    lds_barrier();
  } else {
#pragma unroll
    for (int p = 0; p < kSlots; ++p) issue(ss_of(wave + p * WAVES), p);
  }
  for (int i = 0; i < iters; i += kSlots) {
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      if (i + u >= iters) break;
      __builtin_amdgcn_s_waitcnt(vm_wait((kSlots - 1) * kLoads));
      compute(ss_of(wave + (i + u) * WAVES), u, acc);
      // the slot's reads have returned: the loads write LDS on their own
      __builtin_amdgcn_s_waitcnt(kLgkmWait0);
      issue(ss_of(wave + (i + u + kSlots) * WAVES), u);
    }
  }
  __builtin_amdgcn_s_waitcnt(vm_wait(0));
  __syncthreads();

  i32x4* const red = reinterpret_cast<i32x4*>(lds);          // [WAVES][MT * NT][64]
  static_assert(MT * NT * 1024 <= kSlots * kSlot, "the waves' sums fit the ring");
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[(wave * MT * NT + i * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  // each wave finishes every WAVES-th block of outputs
  for (int b = wave; b < MT * NT; b += WAVES) {
    i32x4 t = red[b * 64 + lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) t += red[(w * MT * NT + b) * 64 + lane];
    const int col = n0 + (b % NT) * 16 + r16;
    if (col >= N) continue;
    const float w_scale = a.ws[col];
    const float bias = a.bias ? bf16_f32(a.bias[col]) : 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = (b / NT) * 16 + 4 * g + r;
      if (row >= M) continue;
      if (gridDim.y > 1) {
        a.part[(size_t)blockIdx.y * partial_slab(M, N) + (size_t)row * N + col] = t[r];
        continue;
      }
      float v = (float)t[r] * ((FUSED ? scales[0] : a.xs[row]) * w_scale);
      if (a.bias) v += bias;
      a.y[(size_t)row * N + col] = f32_bf16(v);
    }
  }
}

template <int MT, int NT, int WAVES, int KW, bool FUSED>
hipError_t launch(const SkinnyArgs& a, const Int8SkinnyPlan& p, hipStream_t stream) {
  hipLaunchKernelGGL((gemm_int8_skinny_kernel<MT, NT, WAVES, KW, FUSED>),
                     dim3((uint32_t)((a.N + 16 * NT - 1) / (16 * NT)), (uint32_t)p.splits), dim3(WAVES * 64), 0, stream,
                     a);
  return hipGetLastError();
}

SkinnyArgs args_of(const void* x, const float* xs, const int8_t* wq, const float* ws, const uint16_t* bias,
                   uint16_t* y, int64_t m, int64_t n, int64_t k, void* workspace, const Int8SkinnyPlan& p) {
  return SkinnyArgs{x, xs, wq, ws, bias, y, static_cast<int32_t*>(workspace), (int)m, (int)n, (int)k, p.k_split};
}

}  // namespace

size_t int8_skinny_bytes(int64_t m, int64_t n, int64_t k) {
  const Int8SkinnyPlan p = plan_skinny8(m, n, k);
  return p.splits > 1 ? round_up((size_t)p.splits * partial_slab(m, n) * sizeof(int32_t), kWorkspaceAlign) : 0;
}

hipError_t launch_int8_skinny(const int8_t* xq, const float* xs, const int8_t* wq, const float* ws,
                              const uint16_t* bias, uint16_t* y, int64_t m, int64_t n, int64_t k, void* workspace,
                              hipStream_t stream) {
  const Int8SkinnyPlan p = plan_skinny8(m, n, k);
  const SkinnyArgs a = args_of(xq, xs, wq, ws, bias, y, m, n, k, workspace, p);
  const hipError_t e = m > 16 ? p.few ? launch<2, 1, 4, 128, false>(a, p, stream) : launch<2, 2, 2, 256, false>(a, p, stream)
                       : p.few ? launch<1, 1, 8, 128, false>(a, p, stream)
                       : m > 1 ? launch<1, 2, 4, 128, false>(a, p, stream)
                               : launch<1, 1, 4, 256, false>(a, p, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_int8_join(a.part, xs, ws, bias, y, p.splits, m, n, stream);
}

hipError_t launch_int8_skinny_bf16(const uint16_t* x, const int8_t* wq, const float* ws, const uint16_t* bias,
                                   uint16_t* y, int64_t n, int64_t k, hipStream_t stream) {
  const Int8SkinnyPlan p = plan_skinny8(1, n, k);
  const SkinnyArgs a = args_of(x, nullptr, wq, ws, bias, y, 1, n, k, nullptr, p);
  return p.few ? launch<1, 1, 8, 128, true>(a, p, stream) : launch<1, 1, 4, 256, true>(a, p, stream);
}

}  // namespace fp8bl
