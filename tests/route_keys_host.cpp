// Prints, for each line "bits number" on standard input, the float's key with its last bits written over
// by ones, and the bits of the float that it stands for.
#include <cinttypes>
#include <cstdio>

#include "route_keys.hpp"

int main() {
  uint32_t bits, number;
  while (std::scanf("%" SCNu32 " %" SCNu32, &bits, &number) == 2) {
    const uint32_t key = tbe::key_of_float(bits) | number;
    std::printf("%" PRIu32 " %" PRIu32 "\n", key, tbe::float_of_key(key, number));
  }
}
