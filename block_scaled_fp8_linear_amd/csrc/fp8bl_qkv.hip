// C ABI from the QKV projection to its cache (declared in include/fp8bl_qkv.h):
// argument validation before any HIP call, and the launches. Nothing here
// touches tensor data.
#include "fp8bl_qkv.h"

#include <cmath>

#include "fp8bl_arrays.h"
#include "fp8bl_ops.h"

namespace {

using namespace fp8bl::checks;
using fp8bl::gate_current_device;
using fp8bl::kWorkspaceAlign;

constexpr int64_t kMaxHeads = 4096;
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxStoreTokens = 65536;   // each token looks for a later one with its slot

// One array of a call in bytes: a view of tokens with a stride, or a plain
// array (token_bytes 0).
struct View {
  const void* p;
  size_t extent;       // from the first byte to the last
  size_t stride;       // between tokens
  size_t row;          // of one token
  uintptr_t align;
  bool out;
  int64_t head_stride;
  int tag;             // an output may be the input of its own tag, strides and all
};

View plain(const void* p, size_t bytes, uintptr_t align, bool out) { return View{p, bytes, 0, 0, align, out, 0, 0}; }

// A view of `heads` heads, checked for itself: its strides, and that an
// output's elements are distinct.
int heads_view(const fp8bl_heads& h, int64_t tokens, int64_t heads, int64_t dim, bool out, int tag, View* v) {
  if (tokens == 0 || heads == 0) {
    *v = plain(nullptr, 0, 16, out);
    return FP8BL_OK;
  }
  // an axis of one element has no stride
  const int64_t ts = tokens == 1 ? 0 : h.token_stride, hs = heads == 1 ? 0 : h.head_stride;
  if (ts < 0 || hs < 0 || ts > kMaxStride || hs > kMaxStride || ts % 8 != 0 || hs % 8 != 0) return FP8BL_INVALID_ARG;
  // below 2^31 2^40 elements of two bytes and 2^12 2^40 more
  const __int128 last = (__int128)(tokens - 1) * ts + (__int128)(heads - 1) * hs + dim;
  if (last >= (__int128)1 << 60) return FP8BL_INVALID_ARG;
  if (out) {
    const bool by_token = (heads == 1 || hs >= dim) && (tokens == 1 || ts >= (heads - 1) * hs + dim);
    const bool by_head = (tokens == 1 || ts >= dim) && (heads == 1 || (__int128)hs >= (__int128)(tokens - 1) * ts + dim);
    if (!by_token && !by_head) return FP8BL_INVALID_ARG;
  }
  const size_t row = ((size_t)(heads - 1) * hs + dim) * 2;
  *v = View{h.data, (size_t)last * 2, (size_t)ts * 2, row, 16, out, hs, tag};
  return FP8BL_OK;
}

// Whether two arrays share a byte. Views with one token stride may lie beside
// each other within it.
bool shared(const View& a, const View& b) {
  if (!overlap(a.p, a.extent, b.p, b.extent)) return false;
  if (a.stride == 0 || a.stride != b.stride) return true;
  if (a.row > a.stride || b.row > a.stride) return true;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const View &lo = pa <= pb ? a : b, &hi = pa <= pb ? b : a;
  const size_t off = (pa <= pb ? pb - pa : pa - pb) % a.stride;
  return off < lo.row || off + hi.row > a.stride;
}

int check_views(const View* v, int count) {
  for (int i = 0; i < count; ++i)
    if (v[i].extent > 0 && v[i].p == nullptr) return FP8BL_INVALID_ARG;
  for (int i = 0; i < count; ++i)
    if (v[i].extent > 0 && !aligned(v[i].p, v[i].align)) return FP8BL_ALIGNMENT;
  for (int i = 0; i < count; ++i)
    for (int j = i + 1; j < count; ++j) {
      const View &a = v[i], &b = v[j];
      if (a.extent == 0 || b.extent == 0 || !(a.out || b.out)) continue;
      if (a.out != b.out && a.tag != 0 && a.tag == b.tag && a.p == b.p && a.stride == b.stride &&
          a.head_stride == b.head_stride && a.extent == b.extent)
        continue;      // in place
      if (shared(a, b)) return FP8BL_INVALID_ARG;
    }
  return FP8BL_OK;
}

struct Views {
  View v[20];
  int count = 0;
  int status = FP8BL_OK;
  void add(const View& x) { v[count++] = x; }
  void heads(const fp8bl_heads& h, const fp8bl_qkv& a, int64_t n, bool out, int tag = 0) {
    View x;
    const int st = heads_view(h, a.tokens, n, a.head_dim, out, tag, &x);
    if (st != FP8BL_OK) status = st;
    else add(x);
  }
  int check() const { return status != FP8BL_OK ? status : check_views(v, count); }
};

int check_sizes(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim) {
  if (tokens < 0 || tokens >= kMaxDim || q_heads < 0 || q_heads > kMaxHeads || k_heads < 0 || k_heads > kMaxHeads)
    return FP8BL_INVALID_ARG;
  return dim < 16 || dim > 256 || dim % 8 != 0 ? FP8BL_INVALID_ARG : FP8BL_OK;
}

int check_turn(const fp8bl_qkv& a) {
  if (a.axes < 1 || a.axes > FP8BL_MAX_AXES || a.interleaved < 0 || a.interleaved > 1) return FP8BL_INVALID_ARG;
  if (a.pairs < 1 || a.pairs > a.head_dim / 2 || a.pairs % (a.interleaved ? 4 : 8) != 0) return FP8BL_INVALID_ARG;
  if (!(a.eps >= 0.0) || !std::isfinite((float)a.eps)) return FP8BL_INVALID_ARG;
  for (int64_t i = 0; i < a.pairs; ++i)
    if (a.axis[i] >= a.axes) return FP8BL_INVALID_ARG;
  return FP8BL_OK;
}

// The arrays of norm and rotation besides the heads.
void turn_views(Views& s, const fp8bl_qkv& a) {
  s.add(plain(a.q_weight, a.q_heads > 0 ? (size_t)a.head_dim * 2 : 0, 16, false));
  s.add(plain(a.k_weight, a.k_heads > 0 ? (size_t)a.head_dim * 2 : 0, 16, false));
  s.add(plain(a.positions, (size_t)a.axes * a.tokens * 4, 4, false));
  s.add(plain(a.inv_freq, (size_t)a.pairs * 4, 4, false));
}

int check_cache(const fp8bl_qkv& a) {
  if (a.cache_rows < 0 || a.cache_rows >= kMaxDim) return FP8BL_INVALID_ARG;
  return FP8BL_OK;
}

void cache_views(Views& s, const fp8bl_qkv& a, bool out) {
  const size_t codes = (size_t)a.cache_rows * a.k_heads * a.head_dim, scales = (size_t)a.cache_rows * a.k_heads * 4;
  s.add(plain(a.slots, a.k_heads > 0 ? (size_t)a.tokens * 4 : 0, 4, false));
  s.add(plain(a.k_cache, codes, 16, out));
  s.add(plain(a.v_cache, codes, 16, out));
  s.add(plain(a.k_scale, scales, 4, out));
  s.add(plain(a.v_scale, scales, 4, out));
}

}  // namespace

FP8BL_EXPORT int fp8_qk_norm_rope(const fp8bl_qkv* args, hipStream_t stream) {
  if (args == nullptr) return FP8BL_INVALID_ARG;
  const fp8bl_qkv& a = *args;
  int st = check_sizes(a.tokens, a.q_heads, a.k_heads, a.head_dim);
  if (st == FP8BL_OK) st = check_turn(a);
  if (st != FP8BL_OK) return st;
  if (a.tokens == 0 || a.q_heads + a.k_heads == 0) return FP8BL_OK;
  Views s;
  s.heads(a.q, a, a.q_heads, false, 1);
  s.heads(a.k, a, a.k_heads, false, 2);
  s.heads(a.q_out, a, a.q_heads, true, 1);
  s.heads(a.k_out, a, a.k_heads, true, 2);
  turn_views(s, a);
  st = s.check();
  if (st == FP8BL_OK) st = gate_current_device();
  return st != FP8BL_OK ? st : hip_status(fp8bl::launch_qk_norm_rope(a, stream));
}

FP8BL_EXPORT size_t fp8_qk_norm_rope_backward_workspace_size(int64_t tokens, int64_t q_heads, int64_t k_heads,
                                                             int64_t head_dim) {
  if (check_sizes(tokens, q_heads, k_heads, head_dim) != FP8BL_OK || tokens == 0 || q_heads + k_heads == 0) return 0;
  return fp8bl::qk_backward_bytes(tokens, q_heads, k_heads, head_dim);
}

FP8BL_EXPORT int fp8_qk_norm_rope_backward(const fp8bl_qkv* args, void* workspace, size_t workspace_bytes,
                                           hipStream_t stream) {
  if (args == nullptr) return FP8BL_INVALID_ARG;
  const fp8bl_qkv& a = *args;
  int st = check_sizes(a.tokens, a.q_heads, a.k_heads, a.head_dim);
  if (st == FP8BL_OK) st = check_turn(a);
  if (st != FP8BL_OK) return st;
  const size_t need = fp8_qk_norm_rope_backward_workspace_size(a.tokens, a.q_heads, a.k_heads, a.head_dim);
  Views s;
  s.heads(a.q, a, a.q_heads, false);
  s.heads(a.k, a, a.k_heads, false);
  s.heads(a.dq, a, a.q_heads, false, 1);
  s.heads(a.dk, a, a.k_heads, false, 2);
  s.heads(a.q_out, a, a.q_heads, true, 1);
  s.heads(a.k_out, a, a.k_heads, true, 2);
  s.add(plain(a.dq_weight, a.dq_weight ? (size_t)a.head_dim * 4 : 0, 4, true));
  s.add(plain(a.dk_weight, a.dk_weight ? (size_t)a.head_dim * 4 : 0, 4, true));
  if (need > 0) turn_views(s, a);
  st = s.check();
  if (st != FP8BL_OK) return st;
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return FP8BL_WORKSPACE;
    if (!aligned(workspace, kWorkspaceAlign)) return FP8BL_ALIGNMENT;
    for (int i = 0; i < s.count; ++i)
      if (s.v[i].extent > 0 && overlap(workspace, need, s.v[i].p, s.v[i].extent)) return FP8BL_INVALID_ARG;
  }
  if (need == 0 && a.dq_weight == nullptr && a.dk_weight == nullptr) return FP8BL_OK;
  st = gate_current_device();
  if (st != FP8BL_OK) return st;
  if (need == 0) {       // empty sums are zeros
    for (float* dw : {a.dq_weight, a.dk_weight})
      if (dw != nullptr && fp8bl::launch_fill_zero(dw, (size_t)a.head_dim * 4, stream) != hipSuccess)
        return FP8BL_HIP_ERROR;
    return FP8BL_OK;
  }
  return hip_status(fp8bl::launch_qk_norm_rope_backward(a, static_cast<float*>(workspace), stream));
}

FP8BL_EXPORT int fp8_kv_store(const fp8bl_qkv* args, hipStream_t stream) {
  if (args == nullptr) return FP8BL_INVALID_ARG;
  const fp8bl_qkv& a = *args;
  int st = check_sizes(a.tokens, 0, a.k_heads, a.head_dim);
  if (st == FP8BL_OK) st = check_cache(a);
  if (st != FP8BL_OK) return st;
  if (a.tokens > kMaxStoreTokens) return FP8BL_INVALID_ARG;
  if (a.tokens == 0 || a.k_heads == 0) return FP8BL_OK;
  Views s;
  s.heads(a.k, a, a.k_heads, false);
  s.heads(a.v, a, a.k_heads, false);
  cache_views(s, a, true);
  st = s.check();
  if (st == FP8BL_OK) st = gate_current_device();
  return st != FP8BL_OK ? st : hip_status(fp8bl::launch_kv_store(a, stream));
}

FP8BL_EXPORT int fp8_kv_load(const fp8bl_qkv* args, hipStream_t stream) {
  if (args == nullptr) return FP8BL_INVALID_ARG;
  const fp8bl_qkv& a = *args;
  int st = check_sizes(a.tokens, 0, a.k_heads, a.head_dim);
  if (st == FP8BL_OK) st = check_cache(a);
  if (st != FP8BL_OK) return st;
  if (a.tokens == 0 || a.k_heads == 0) return FP8BL_OK;
  Views s;
  s.heads(a.k_out, a, a.k_heads, true);
  s.heads(a.v_out, a, a.k_heads, true);
  cache_views(s, a, false);
  st = s.check();
  if (st == FP8BL_OK) st = gate_current_device();
  return st != FP8BL_OK ? st : hip_status(fp8bl::launch_kv_load(a, stream));
}

FP8BL_EXPORT int fp8_qk_norm_rope_store(const fp8bl_qkv* args, hipStream_t stream) {
  if (args == nullptr) return FP8BL_INVALID_ARG;
  const fp8bl_qkv& a = *args;
  int st = check_sizes(a.tokens, a.q_heads, a.k_heads, a.head_dim);
  if (st == FP8BL_OK) st = check_turn(a);
  if (st == FP8BL_OK) st = check_cache(a);
  if (st != FP8BL_OK) return st;
  if (a.tokens > kMaxStoreTokens) return FP8BL_INVALID_ARG;
  if (a.tokens == 0 || a.q_heads + a.k_heads == 0) return FP8BL_OK;
  Views s;
  s.heads(a.q, a, a.q_heads, false, 1);
  s.heads(a.k, a, a.k_heads, false);
  s.heads(a.v, a, a.k_heads, false);
  s.heads(a.q_out, a, a.q_heads, true, 1);
  turn_views(s, a);
  cache_views(s, a, true);
  st = s.check();
  if (st == FP8BL_OK) st = gate_current_device();
  return st != FP8BL_OK ? st : hip_status(fp8bl::launch_qk_norm_rope_store(a, stream));
}
