// Host-side argument checks shared by the C entry points (not installed).
#pragma once

#include "kvc_internal.h"

namespace kvc {

struct Range {
  const void* p;
  size_t n;
};

inline bool overlap(Range a, Range b) {
  if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = uintptr_t(a.p), b0 = uintptr_t(b.p);
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

// Every output must be disjoint from every input and from every other output.
inline bool any_alias(const Range* in, int n_in, const Range* out, int n_out) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(out[i], in[j])) return true;
    for (int j = i + 1; j < n_out; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

inline bool aligned(const void* p, size_t a) { return (uintptr_t(p) & (a - 1)) == 0; }

inline int launch_status(hipError_t e) {
  if (e != hipSuccess) return KVC_EDEVICE;
  return hipGetLastError() == hipSuccess ? KVC_OK : KVC_EDEVICE;
}

}  // namespace kvc
