// What the host code of the language-model products (lm.hip, q4.hip) shares: limits of
// sizes, integer helpers, and the device's compute units.  Plain C++.
#pragma once

#include <climits>
#include <cstdint>

namespace sgemm {
namespace lm {

// Largest extent taken: tile edges past the end of a matrix stay within int.
constexpr int kMostExtent = INT_MAX - 1024;

// Most workgroups of 256 a launch takes along x: below 2^32 work items.
constexpr int kMostBlocks = (1 << 24) - 1;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
inline bool aligned(const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Compute units of the current device (cached; 0 on failure, with the error in *rc).
// Defined in lm.hip.
int compute_units(int *rc);

}  // namespace lm
}  // namespace sgemm
