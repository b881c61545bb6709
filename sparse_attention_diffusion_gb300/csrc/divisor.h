// Division by a divisor known at launch.
#pragma once
#include <cstdint>

namespace mcs {

// Of n < 2^31: with l = ceil(log2 d) and m = floor(2^(31 + l) / d) + 1,
// n / d = (n m) >> (31 + l) (Granlund and Montgomery).
struct Divisor {
  uint32_t mul = 0;
  int shift = 0;
  Divisor() = default;
  explicit Divisor(int d) {
    int l = 0;
    while ((1ll << l) < d) ++l;
    mul = uint32_t((1ull << (31 + l)) / uint32_t(d) + 1);
    shift = 31 + l;
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int div(int n) const { return int((uint64_t(uint32_t(n)) * mul) >> shift); }
#endif
};

}  // namespace mcs
