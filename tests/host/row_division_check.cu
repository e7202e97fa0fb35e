// Host-only check of the row attention kernel's division of a row index by the
// query heads per KV head (no GPU): exact for every divisor and row tried, up
// to the ends of both, also where the multiplied reciprocal alone is one too
// large. Compiled and run by tests/test_rows_division.py.
#include <cstdio>
#include <initializer_list>

#include "row_division.h"

int main() {
  long long bad = 0, alone = 0, tried = 0;
  auto one = [&](uint32_t d, uint64_t x) {
    if (x > 0xffffffffull) return;
    const kv2::RowDivision by = kv2::row_division(d);
    ++tried;
    if (by(uint32_t(x)) != uint32_t(x) / d) {
      if (bad++ < 10) std::printf("FAIL %llu / %u\n", (unsigned long long)x, d);
    }
    if (d > 1 && uint32_t((x * by.inv) >> 32) != uint32_t(x) / d) ++alone;
  };
  auto all = [&](uint32_t d) {
    for (uint64_t x = 0; x < 600; ++x) one(d, x);
    for (int b = 10; b <= 32; ++b)
      for (long long o = -3; o <= 3; ++o) {
        const uint64_t k = ((uint64_t(1) << b) / d) * d;              // around multiples of d
        one(d, uint64_t((long long)k + o < 0 ? 0 : (long long)k + o));
        one(d, (uint64_t(1) << b) + uint64_t(o));
      }
  };
  for (uint32_t d = 1; d < 3000; ++d) all(d);
  for (uint32_t d : {46341u, 50000u, 65535u, 65536u, 65537u, 131070u, (1u << 30) - 1u, 1u << 30}) all(d);
  one(1000, 6100999);
  one(65535, 131069);
  std::printf("%lld quotients, %lld wrong, %lld where the product alone is\n", tried, bad, alone);
  return bad != 0 || alone == 0;
}
