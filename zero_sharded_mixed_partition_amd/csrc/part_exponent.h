// The power of two that a part of X X^T is scaled by (orthogonalize_thin.hip): an
// exponent of its elements, or one of two marks.
#pragma once
#include <climits>

namespace zero_shard {

constexpr int kAllZero = INT_MIN / 4;            // no element but zeros so far
constexpr int kNotFinite = INT_MAX;              // an inf or a NaN

constexpr bool has_exponent(int e) { return e >= INT_MIN / 8; }

// The power of two that takes a part's sums to the scale of the parts' largest
// exponent; 0 for a part of zeros.  Not to be formed where the largest is kNotFinite.
constexpr int part_shift(int e, int top) { return has_exponent(e) ? 2 * (e - top) : 0; }

}  // namespace zero_shard
