// packed_tile.cuh — fp16x2 arithmetic that turns packed INT2 codes into
// tensor-core operands, and the operand tile addressing shared by the tcgen05
// attention kernels.
#pragma once

#include "common.cuh"

namespace kv2 {

// byte offset of 16-byte chunk `c` (0, 1) of row `row` in a no-swizzle
// [row/8][2][8][16 B] operand tile (K = 16 columns of 16-bit values)
__device__ __forceinline__ uint32_t nosw_off(int row, int c) {
  return uint32_t((row >> 3) * 256 + c * 128 + (row & 7) * 16);
}

// two fp32 -> packed bf16x2 / f16x2 (one paired conversion, round to nearest even)
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// d = a * b + c on two fp16 lanes; d = a + b
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The codes of channels 2i, 2i+1 of an 8-channel chunk sit at bits 4i and
// 4i+2 of its 16-bit code field. With the field in both halves of x (and x
// shifted right by 8 for i >= 2), (x & mask) | 0x6400 puts the fp16 numbers
// 1024 + code * 16^i' in the low half and 1024 + 4 code * 16^i' in the high
// half (i' = i mod 2, bits within the fp16 mantissa); one fp16 fma with the
// exact constants below leaves the two codes (exact small integers).
__device__ __forceinline__ uint32_t code_pair_f16(uint32_t x, uint32_t x8, int i) {
  const uint32_t src = (i < 2) ? x : x8;
  const int ip = i & 1;
  const uint32_t mask = (3u << (4 * ip)) | (3u << (16 + 4 * ip + 2));
  const uint32_t scale = ip ? 0x24002C00u : 0x34003C00u;    // {1/16, 1/64} : {1, 1/4}
  const uint32_t offset = ip ? 0xCC00D400u : 0xDC00E400u;   // {-64, -16} : {-1024, -256}
  return hfma2((src & mask) | 0x64006400u, scale, offset);
}
// the 16-bit code field `lc & 1` of word w in both halves of a word
__device__ __forceinline__ uint32_t field_both(uint32_t w, int lc) {
  return __byte_perm(w, 0u, (lc & 1) ? 0x3232u : 0x1010u);
}

}  // namespace kv2
