// divide.hpp -- division by a number known at launch, as a product.
#pragma once

#include <stdint.h>

namespace is {

// n / d for 0 <= n < 2^31 by a product: with 2^(s - 1) < d <= 2^s and
// m = ceil(2^(31 + s) / d), n m >> 31 + s is exact. (The index arithmetic of a
// workgroup would otherwise spend several divisions before its first load.)
struct Divisor {
  unsigned m, s;
};
inline Divisor divisor(unsigned d) {
  unsigned s = 0;
  while (((uint64_t)1 << s) < d) ++s;
  return {(unsigned)((((uint64_t)1 << (31 + s)) + d - 1) / d), s};
}
__device__ __forceinline__ int divide(int n, Divisor d) {
  return (int)(((uint64_t)(unsigned)n * d.m) >> (31 + d.s));
}

}  // namespace is
