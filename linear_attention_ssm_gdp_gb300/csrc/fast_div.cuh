// Division by a number that the launch knows: one high product, one sum and a shift.
#pragma once

#include <stdint.h>

namespace gdp {

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31: with l = ceil(log2 d) and mul = floor(2^32 (2^l - d) / d) + 1 the
// quotient is (high half of n mul, plus n) / 2^l (Granlund and Montgomery).
struct Div {
  uint32_t d, mul, shift;
};
inline Div div_by(uint32_t d) {
  uint32_t l = 0;
  while (l < 32 && (1ull << l) < d) ++l;
  const uint64_t m = (((1ull << l) - d) << 32) / d + 1;
  return {d, (uint32_t)m, l};
}
__device__ __forceinline__ uint32_t quot(uint32_t n, const Div& v) {
  return (uint32_t)(((uint64_t)__umulhi(n, v.mul) + n) >> v.shift);
}

}  // namespace gdp
