// row_division.h — the quotient of a row index by the query heads per KV head.
#pragma once

#include <cstdint>

namespace kv2 {

// floor(x / d) for every x below 2^32. With inv = ceil(2^32 / d) and
// e = inv d - 2^32 < d, x inv / 2^32 = x / d + x e / (d 2^32), which is less
// than one too large: the product's high half is the quotient or one more, and
// a comparison says which. (Without it the quotient is only right while x e is
// below 2^32.)
struct RowDivision {
  uint32_t d = 1, inv = 0;     // inv 0: d = 1
#ifdef __CUDACC__
  __host__ __device__ __forceinline__
#endif
  uint32_t operator()(uint32_t x) const {
    if (inv == 0) return x;
    const uint32_t q = uint32_t((uint64_t(x) * inv) >> 32);
    return q - (uint64_t(q) * d > x ? 1u : 0u);
  }
};

inline RowDivision row_division(uint32_t d) {
  RowDivision r;
  r.d = d;
  r.inv = d > 1 ? uint32_t(((uint64_t(1) << 32) + d - 1) / d) : 0;
  return r;
}

}  // namespace kv2
