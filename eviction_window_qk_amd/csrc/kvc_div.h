// Quotients by divisors known at launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kvc {

// Quotient by a divisor known at launch: q = (mulhi(x, m) + x) >> s, exact for
// 0 <= x < 2^31 (m = floor(2^32 (2^s - d) / d) + 1, s = ceil(log2 d)); Granlund and
// Montgomery, Division by Invariant Integers using Multiplication, 1994.
struct FastDiv {
  uint32_t d, m, s;
};

inline FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  const uint64_t m = ((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1;
  return FastDiv{d, uint32_t(m), s};
}

__host__ __device__ __forceinline__ uint32_t quot(FastDiv f, uint32_t x) {
  return uint32_t(((uint64_t(x) * f.m) >> 32) + x) >> f.s;
}

// The same for any 32-bit x.
__device__ __forceinline__ uint32_t quot32(FastDiv f, uint32_t x) {
  const uint32_t hi = __umulhi(x, f.m);
  return f.s == 0 ? x : (((x - hi) >> 1) + hi) >> (f.s - 1);
}

}  // namespace kvc
