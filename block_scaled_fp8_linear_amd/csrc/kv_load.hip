// Rows of the E4M3 cache back as bf16(fl32(code * S)); zeros for a token whose
// slot is outside the cache. A wave takes a token, 64 / L heads of its keys and
// values at a time; three bytes an element in all, no other work to speak of, and
// bound by them: 131071 rows of 8 heads of 128 take 137 us (5.9 TB/s), 129 rows
// 3.2, a launch's own time.
#include "fp8bl_ops.h"
#include "qkv_device.h"

namespace fp8bl {

namespace {

struct LoadArgs {
  const int32_t* slots;
  const uint8_t* codes[2];     // keys, values
  const float* scales[2];
  HeadView out[2];
  int tokens, dim, rows;
};

template <int L, bool PAST>
__global__ __launch_bounds__(kQkvThreads)
void load_kernel(LoadArgs g) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = 8 * (lane % L), heads = g.out[0].heads;
  for (int64_t token = (int64_t)blockIdx.x * kQkvWaves + wave; token < g.tokens;
       token += (int64_t)gridDim.x * kQkvWaves) {
    const int slot = g.slots[token];
    const bool kept = slot >= 0 && slot < g.rows;
    for (int h = lane / L; h < heads; h += 64 / L) {
      if (col >= g.dim) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        u32x4 out = {0, 0, 0, 0};
        if (kept) {
          const size_t row = (size_t)slot * heads + h;
          const u32x2* const from = reinterpret_cast<const u32x2*>(g.codes[i] + row * g.dim + col);
          const u32x2 codes = PAST ? __builtin_nontemporal_load(from) : *from;
          const float s = g.scales[i][row];
          const u32x2 a = dequant4(codes[0], s), b = dequant4(codes[1], s);
          out = u32x4{a[0], a[1], b[0], b[1]};
        }
        put8<PAST>(g.out[i].p + token * g.out[i].ts + h * g.out[i].hs + col, out);
      }
    }
  }
}

struct Load {
  const fp8bl_qkv& a;
  hipStream_t stream;
  template <int L>
  hipError_t run() {
    const LoadArgs g{a.slots,
                     {a.k_cache, a.v_cache},
                     {a.k_scale, a.v_scale},
                     {head_view(a.k_out, a.k_heads), head_view(a.v_out, a.k_heads)},
                     (int)a.tokens,
                     (int)a.head_dim,
                     (int)a.cache_rows};
    const int64_t blocks = (a.tokens + kQkvWaves - 1) / kQkvWaves;
    const dim3 grid((uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks));
    if (past_caches(a.tokens * a.k_heads * a.head_dim * 6))       // of keys and values one byte and two each
      hipLaunchKernelGGL((load_kernel<L, true>), grid, dim3(kQkvThreads), 0, stream, g);
    else
      hipLaunchKernelGGL((load_kernel<L, false>), grid, dim3(kQkvThreads), 0, stream, g);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_kv_load(const fp8bl_qkv& a, hipStream_t stream) { return with_lanes(a.head_dim, Load{a, stream}); }

}  // namespace fp8bl
