// route_keys.hpp -- floats as whole numbers in the same order, whose last bits a number is
// written over.  Plain C++, which compiles for a CPU alone too; floats are given by their bits.
#pragma once

#include <cstdint>

namespace tbe {

// The keys of finite floats, of -FLT_MAX and above; -infinity's is 1 below, and 0 is none's.
constexpr uint32_t kFirstFiniteKey = 0x00800000u;

// No NaN and no -0.
constexpr uint32_t key_of_float(uint32_t bits) {
  return bits ^ (bits >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}

// The float whose key it is, down to the bits `number` that are written over.  -infinity's key
// has a mantissa of ones once inverted, so that it would come back as a NaN.
constexpr uint32_t float_of_key(uint32_t key, uint32_t number) {
  if (key < kFirstFiniteKey) return 0xFF800000u;
  const uint32_t bits = key & ~number;
  return bits ^ (bits >> 31 ? 0x80000000u : 0xFFFFFFFFu);
}

}  // namespace tbe
