// Division by a number that a launch fixes.
#pragma once

#include <cstdint>

namespace ra {

// Quotients by a fixed d of n < 2^25: mul = ceil(2^(25 + l) / d) with
// 2^(l - 1) < d <= 2^l is off by less than d / d, so n * mul / 2^(25 + l) is off
// by less than n 2^l / d / 2^(25 + l) < 1 / d and has the quotient's floor. (Two
// runtime divisions a thread were a third of the instructions.)
struct Divisor {
  uint32_t d, mul;
  int shift;
  explicit Divisor(uint32_t d_) : d(d_) {
    int l = 0;
    while ((1ull << l) < d) ++l;
    shift = 25 + l;
    mul = (uint32_t)(((1ull << shift) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t of(uint32_t n) const {
    return (uint32_t)(((uint64_t)n * mul) >> shift);
  }
};

}  // namespace ra
