// The arrays of a call as the ABI files check them: present, aligned, and no
// output over another array (host only, no HIP calls).
#pragma once

#include <initializer_list>

#include "fp8bl_checks.h"
#include "fp8bl_internal.h"

namespace fp8bl {
namespace checks {

// One array of a call: `bytes` 0 where it is empty or not given (optional).
struct Array {
  const void* p;
  size_t bytes;
  uintptr_t align;
  bool out;
  const void* same = nullptr;   // an output it may coincide with exactly
};

inline int check_arrays(std::initializer_list<Array> arrays) {
  for (const Array& a : arrays)
    if (a.bytes > 0 && a.p == nullptr) return FP8BL_INVALID_ARG;
  for (const Array& a : arrays)
    if (a.bytes > 0 && !aligned(a.p, a.align)) return FP8BL_ALIGNMENT;
  for (const Array* a = arrays.begin(); a != arrays.end(); ++a)
    for (const Array* b = a + 1; b != arrays.end(); ++b) {
      if (a->bytes == 0 || b->bytes == 0 || !(a->out || b->out)) continue;
      if ((a->same != nullptr && a->same == b->p && a->p == b->p) ||
          (b->same != nullptr && b->same == a->p && a->p == b->p))
        continue;
      if (overlap(a->p, a->bytes, b->p, b->bytes)) return FP8BL_INVALID_ARG;
    }
  return FP8BL_OK;
}

// The workspace as one more output, once the arrays themselves are right.
inline int check_workspace(const void* ws, size_t have, size_t need, std::initializer_list<Array> arrays) {
  if (need == 0) return FP8BL_OK;
  if (ws == nullptr || have < need) return FP8BL_WORKSPACE;
  if (!aligned(ws, kWorkspaceAlign)) return FP8BL_ALIGNMENT;
  for (const Array& a : arrays)
    if (a.bytes > 0 && overlap(ws, need, a.p, a.bytes)) return FP8BL_INVALID_ARG;
  return FP8BL_OK;
}

}  // namespace checks
}  // namespace fp8bl
