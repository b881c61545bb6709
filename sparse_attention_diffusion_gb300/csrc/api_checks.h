// Checks of pointers that the C ABI's translation units share.
#pragma once
#include <cstdint>

namespace mcs {

inline bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned16_or_null(const void* p) { return p == nullptr || aligned16(p); }

// Byte ranges, for the refusal of outputs that alias inputs. A null pointer is no range.
struct Range {
  const char* at;
  long long bytes;
};
inline bool overlap(const Range& a, const Range& b) {
  return a.at != nullptr && b.at != nullptr && a.at < b.at + b.bytes && b.at < a.at + a.bytes;
}
inline Range range(const void* p, long long bytes) { return {static_cast<const char*>(p), bytes}; }

}  // namespace mcs
