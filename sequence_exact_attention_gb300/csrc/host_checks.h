// Argument checks on the host that the caches' entry points share.
#pragma once

#include <cstddef>
#include <cstdint>

namespace ra {

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

constexpr long long kMaxElems = 0x7fffffffLL;   // 32-bit sizes of token tensors

// The bytes of one of a call's tensors (none where it is not given).
struct Bytes {
  const void* p;
  size_t n;
};
// Whether two tensors that a call writes, or one that it writes and one that it
// reads, share a byte.
template <size_t kOuts, size_t kIns>
bool overlap(const Bytes (&outs)[kOuts], const Bytes (&ins)[kIns]) {
  auto meet = [](const Bytes& x, const Bytes& y) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    return x.p && y.p && x.n && y.n && a < b + y.n && b < a + x.n;
  };
  for (size_t i = 0; i < kOuts; ++i) {
    for (const Bytes& x : ins)
      if (meet(outs[i], x)) return true;
    for (size_t k = 0; k < i; ++k)
      if (meet(outs[i], outs[k])) return true;
  }
  return false;
}

}  // namespace ra
