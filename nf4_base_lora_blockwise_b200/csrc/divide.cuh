// divide.cuh -- division of 32-bit indices by a divisor that a launch knows, by one high product.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define QLORA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define QLORA_HOST_DEVICE inline
#endif

namespace qlora {

// n / d, exact for n d < 2^32: the multiplier ceil(2^32 / d) is e < d over d too large in 2^32, and the
// quotient right while n e < 2^32.  (Any 31-bit n would take a shift behind the product: rotary
// positions of 16 tokens 1.86 -> 2.13 us, of 4096 packed rows 16.9 -> 17.6.)
struct Divide {
  uint32_t mul, d;
};
inline Divide divide_by(uint32_t d) {
  return {static_cast<uint32_t>((0x100000000ull + d - 1) / d), d};  // (0 for d = 1: see below)
}
QLORA_HOST_DEVICE uint32_t quotient(uint32_t n, Divide v) {
#if defined(__CUDA_ARCH__)
  return v.d == 1 ? n : __umulhi(n, v.mul);
#else
  return v.d == 1 ? n : static_cast<uint32_t>((static_cast<uint64_t>(n) * v.mul) >> 32);
#endif
}
// Heads of d items each whose items n < heads d are all divided by d exactly.
inline int exact_heads(int d) {
  const uint64_t square = static_cast<uint64_t>(d) * static_cast<uint64_t>(d);
  const uint64_t heads = square ? 0x100000000ull / square : 0x7FFFFFFFull;
  return heads < 0x7FFFFFFFull ? static_cast<int>(heads) : 0x7FFFFFFF;
}

}  // namespace qlora
