// swa_turn.h — angles per position as fractions of a turn (host; no CUDA, so
// that a test can compile it alone).
#pragma once
#include <cmath>
#include <cstdint>

namespace swa {

// round(2^64 * (radians / 2 pi mod 1)), exact but for that rounding: 1 / (2 pi)
// as the sum of two doubles, the product with the first split by fma into a
// rounded value and its error.  One double for the product would leave a
// fraction of 2^-53 of the whole turns beside it, which a far position
// multiplies: 3e-3 radians at 2^31 and a frequency of 2^20.  A negative angle is
// the opposite of its positive twin, where 1 - fraction would have lost the
// small one's bits.  |radians| <= 2^20.
inline uint64_t turn_fraction(double radians) {
  constexpr double kHigh = 0.15915494309189535, kLow = -9.839338337591243e-18;  // 1 / (2 pi)
  const double f = std::fabs(radians);
  const double turns = f * kHigh;
  const double rest = std::fma(f, kLow, std::fma(f, kHigh, -turns));
  // in steps of 2^-64 turns: whole ones of the rounded product, then the others
  const double steps = (turns - std::floor(turns)) * 18446744073709551616.0, whole = std::floor(steps);
  const double more = (steps - whole) + rest * 18446744073709551616.0;  // within +-2^30
  const uint64_t n = static_cast<uint64_t>(whole) + static_cast<uint64_t>(static_cast<int64_t>(std::llrint(more)));
  return radians < 0 ? ~n + 1 : n;
}

}  // namespace swa
