// Joins of split partials (fp32 slabs of the split columns) with the layer
// operators' epilogues: the partials are added in split order, then bias, activation,
// residual (or the gate's product) and one rounding of each output. Bound by
// the partials' bytes, or with few rows by the latency of one thread's loads:
// eight splits' loads are in flight at once, and small outputs use narrower
// threads, so that enough of them run. (512 x 5120 with residual: three splits
// 7.4 us, 5.7 TB/s, six splits 11.7 us, 6.3 TB/s.)
#include "fp8bl_act.h"
#include "fp8bl_device.h"
#include "fp8bl_internal.h"

namespace fp8bl {

namespace {

constexpr int kThreads = 256;

template <int VEC>
struct Row {
  float v[VEC];
};

template <int VEC>
__device__ __forceinline__ Row<VEC> load_f32(const float* p) {
  Row<VEC> r;
  if constexpr (VEC == 1) {
    r.v[0] = *p;
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(p + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) r.v[4 * i + e] = a[e];
    }
  }
  return r;
}

template <int VEC>
__device__ __forceinline__ Row<VEC> load_bf16(const uint16_t* p) {
  Row<VEC> r;
  if constexpr (VEC == 1) {
    r.v[0] = bf16_f32(*p);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const u32x2 a = *reinterpret_cast<const u32x2*>(p + 4 * i);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        r.v[4 * i + 2 * e] = __uint_as_float(a[e] << 16);
        r.v[4 * i + 2 * e + 1] = __uint_as_float(a[e] & 0xFFFF0000u);
      }
    }
  }
  return r;
}

template <int VEC>
__device__ __forceinline__ void store_bf16(uint16_t* p, const Row<VEC>& r) {
  if constexpr (VEC == 1) {
    *p = f32_bf16(r.v[0]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const u32x2 a = {pack_bf16x2(r.v[4 * i], r.v[4 * i + 1]), pack_bf16x2(r.v[4 * i + 2], r.v[4 * i + 3])};
      *reinterpret_cast<u32x2*>(p + 4 * i) = a;
    }
  }
}

// Partials p, p + stride, .. (`count` of them), added in order.
template <int VEC>
__device__ __forceinline__ Row<VEC> sum_splits(const float* p, size_t stride, int count) {
  Row<VEC> t = load_f32<VEC>(p);
  int i = 1;
  for (; i + 8 <= count; i += 8) {
    Row<VEC> b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = load_f32<VEC>(p + (size_t)(i + j) * stride);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) t.v[e] += b[j].v[e];
  }
  // the rest, also at once: past the end the last partial is read again and
  // not added
  if (i < count) {
    Row<VEC> b[7];
#pragma unroll
    for (int j = 0; j < 7; ++j) b[j] = load_f32<VEC>(p + (size_t)min(i + j, count - 1) * stride);
#pragma unroll
    for (int j = 0; j < 7; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) t.v[e] = i + j < count ? t.v[e] + b[j].v[e] : t.v[e];
  }
  return t;
}

// Columns c0 .. n of every row (`count` outputs). The partials are [m, n - c0]
// slabs: output f of the columns is element f of each.
template <int ACT, int VEC, bool GLU>
__global__ __launch_bounds__(kThreads)
void join_kernel(const float* __restrict__ part, uint16_t* y, int splits, size_t count, size_t slab,
                 uint32_t n, uint32_t c0, LayerEpilogue ep) {
  const uint32_t width = n - c0;
  for (size_t f = ((size_t)blockIdx.x * kThreads + threadIdx.x) * VEC; f < count;
       f += (size_t)gridDim.x * kThreads * VEC) {
    // (64-bit divisions only where 32 bits do not hold the count)
    const size_t row = count >> 32 ? f / width : (uint32_t)f / width;
    const uint32_t col = c0 + (uint32_t)(f - row * width);
    const size_t i = row * n + col;
    if constexpr (GLU) {
      const Row<VEC> g = sum_splits<VEC>(part + f, 2 * slab, splits);
      const Row<VEC> u = sum_splits<VEC>(part + slab + f, 2 * slab, splits);
      if (ep.g) {
        store_bf16<VEC>(ep.g + i, g);
        store_bf16<VEC>(ep.u + i, u);
      }
      Row<VEC> h;
#pragma unroll
      for (int e = 0; e < VEC; ++e) h.v[e] = act_f32<ACT>(g.v[e]) * u.v[e];
      store_bf16<VEC>(y + i, h);
    } else {
      Row<VEC> res;
      if (ep.residual) res = load_bf16<VEC>(ep.residual + i);
      Row<VEC> t = sum_splits<VEC>(part + f, slab, splits);
      if (ep.bias) {
        const Row<VEC> b = load_bf16<VEC>(ep.bias + col);
#pragma unroll
        for (int e = 0; e < VEC; ++e) t.v[e] += b.v[e];
      }
      if (ep.z) store_bf16<VEC>(ep.z + i, t);
#pragma unroll
      for (int e = 0; e < VEC; ++e) t.v[e] = act_f32<ACT>(t.v[e]);
      if (ep.residual) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) t.v[e] += res.v[e];
      }
      store_bf16<VEC>(y + i, t);
    }
  }
}

template <int VEC, bool GLU>
hipError_t launch(const float* part, uint16_t* y, int splits, int64_t m, int64_t n, int64_t c0,
                  const LayerEpilogue& ep, hipStream_t stream) {
  const size_t count = (size_t)m * (n - c0), blocks = (count + kThreads * VEC - 1) / (kThreads * VEC);
  const dim3 grid((uint32_t)(blocks < (1u << 20) ? blocks : (1u << 20)));
  with_act(ep.act, [&](auto a) {
    hipLaunchKernelGGL((join_kernel<decltype(a)::value, VEC, GLU>), grid, dim3(kThreads), 0, stream, part, y,
                       splits, count, partial_slab((size_t)m, (size_t)(n - c0)), (uint32_t)n, (uint32_t)c0, ep);
  });
  return hipGetLastError();
}

// Four outputs a thread where rows are whole quads and there are enough of
// them for every CU (2^18 outputs are 256 workgroups of quads), else one.
// (c0 is a multiple of 128.)
template <bool GLU>
hipError_t join(const float* part, uint16_t* y, int splits, int64_t m, int64_t n, int64_t c0,
                const LayerEpilogue& ep, hipStream_t stream) {
  if (n % 4 == 0 && m * (n - c0) >= (1 << 18)) return launch<4, GLU>(part, y, splits, m, n, c0, ep, stream);
  return launch<1, GLU>(part, y, splits, m, n, c0, ep, stream);
}

}  // namespace

hipError_t launch_join_layer(const float* part, uint16_t* y, int splits, int64_t m, int64_t n, int64_t c0,
                             const LayerEpilogue& ep, hipStream_t stream) {
  return join<false>(part, y, splits, m, n, c0, ep, stream);
}

hipError_t launch_join_glu(const float* part, uint16_t* h, int splits, int64_t m, int64_t n, int64_t c0,
                           const LayerEpilogue& ep, hipStream_t stream) {
  return join<true>(part, h, splits, m, n, c0, ep, stream);
}

}  // namespace fp8bl
