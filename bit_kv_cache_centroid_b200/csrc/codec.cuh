// codec.cuh — the INT2 coder of 32-channel sub-groups, shared by the append's
// key and value kernels.
#pragma once

#include <cfloat>

#include "common.cuh"
#include "internal.h"

namespace kv2 {

// Codes of the 32 values x of one sub-group with the group's (s, z): the
// quotient (x - z) * inv_s rounded to the nearest integer and clamped to
// 0..3, two channels per packed instruction (each lane rounded as its scalar
// form); bit c of `redo` flags a quotient within 2^-18 of a half-integer
// (|q - rint(q)| > 1/2 - 2^-18), whose code the correctly rounded division
// must decide. With E, also the residual errors x - (code * s + z). A group
// of scale 0 holds x = z only (z is the rounded-down minimum and s the
// rounded-up range / 3): its codes are 0 and its errors x - z whatever the
// quotient gave.
template <bool E>
__device__ __forceinline__ void code32(const float (&x)[kGroup], const GroupParams& gp, float inv_s,
                                       uint32_t& w0, uint32_t& w1, uint32_t& redo, float (&ev)[kGroup]) {
  const f32x2 z2 = pk2(gp.z, gp.z), is2 = pk2(inv_s, inv_s), s2 = pk2(gp.s, gp.s);
  w0 = w1 = redo = 0;
#pragma unroll
  for (int c = 0; c < kGroup; c += 2) {
    const float2 qa = up2(fmul2(fsub2(pk2(x[c], x[c + 1]), z2), is2));
    const float r0 = rintf(qa.x), r1 = rintf(qa.y);
    redo |= (uint32_t(fabsf(__fsub_rn(qa.x, r0)) > 0.5f - 0x1p-18f) << c) |
            (uint32_t(fabsf(__fsub_rn(qa.y, r1)) > 0.5f - 0x1p-18f) << (c + 1));
    const float c0 = fminf(fmaxf(r0, 0.0f), 3.0f), c1 = fminf(fmaxf(r1, 0.0f), 3.0f);
    const uint32_t q = uint32_t(c0) | (uint32_t(c1) << 2);
    if (c < 16) w0 |= q << (2 * c); else w1 |= q << (2 * (c - 16));
    if constexpr (E) {
      const float2 e = up2(fsub2(pk2(x[c], x[c + 1]), ffma2(pk2(c0, c1), s2, z2)));
      ev[c] = e.x;
      ev[c + 1] = e.y;
    }
  }
  if (gp.s == 0.0f) w0 = w1 = redo = 0;
}

// Codes of the 32 values (bf16) at vrow; a group of GS channels spans GS / 32
// consecutive lanes, which share its range by shuffles (every lane of the warp
// takes part).
template <int GS>
__device__ __forceinline__ GroupParams code_values(const uint16_t* vrow, uint32_t& w0, uint32_t& w1) {
  constexpr int SPG = GS / kGroup;
  float x[kGroup];
#pragma unroll
  for (int c8 = 0; c8 < kGroup / 8; ++c8) {
    const uint4 vv = *reinterpret_cast<const uint4*>(vrow + c8 * 8);
    const uint32_t vu[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      x[c8 * 8 + 2 * q] = __uint_as_float(vu[q] << 16);
      x[c8 * 8 + 2 * q + 1] = __uint_as_float(vu[q] & 0xffff0000u);
    }
  }
  float mn = x[0], mx = x[0];
#pragma unroll
  for (int c = 1; c + 1 < kGroup; c += 2) { mn = fmin3(mn, x[c], x[c + 1]); mx = fmax3(mx, x[c], x[c + 1]); }
  mn = fminf(mn, x[kGroup - 1]);
  mx = fmaxf(mx, x[kGroup - 1]);
#pragma unroll
  for (int o = 1; o < SPG; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  const GroupParams gp = group_params(mn, mx);
  const float inv_s = __frcp_rn(gp.s);
  uint32_t redo;
  float unused[kGroup];
  code32<false>(x, gp, inv_s, w0, w1, redo, unused);
  // the rare channels whose code the correctly rounded division decides
#pragma unroll 1
  for (; redo; redo &= redo - 1) {
    const int c = __ffs(redo) - 1;
    const uint32_t q = group_code(__uint_as_float(uint32_t(vrow[c]) << 16), gp);
    if (c < 16) w0 = (w0 & ~(3u << (2 * c))) | (q << (2 * c));
    else w1 = (w1 & ~(3u << (2 * (c - 16)))) | (q << (2 * (c - 16)));
  }
  return gp;
}

// The same codes by GS / 8 consecutive lanes, 8 values each: returns this
// lane's 16 bits of the code words. The minimum, the maximum and the choice of
// each code are those of code_values, whatever lanes share them. Lanes move 16
// contiguous bytes and hold 8 values, a quarter of code_values' registers.
template <int GS>
__device__ __forceinline__ GroupParams code_values8(const uint4 vv, uint32_t& bits) {
  const uint32_t vu[4] = {vv.x, vv.y, vv.z, vv.w};
  float x[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    x[2 * q] = __uint_as_float(vu[q] << 16);
    x[2 * q + 1] = __uint_as_float(vu[q] & 0xffff0000u);
  }
  float mn = fminf(fmin3(x[0], x[1], x[2]), fmin3(x[3], x[4], x[5])), mx = fmaxf(fmax3(x[0], x[1], x[2]), fmax3(x[3], x[4], x[5]));
  mn = fmin3(mn, x[6], x[7]);
  mx = fmax3(mx, x[6], x[7]);
#pragma unroll
  for (int o = 1; o < GS / 8; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  const GroupParams gp = group_params(mn, mx);
  const float inv_s = __frcp_rn(gp.s);
  uint32_t redo = 0;
  bits = 0;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float q = __fmul_rn(__fsub_rn(x[c], gp.z), inv_s), r = rintf(q);
    bits |= uint32_t(fminf(fmaxf(r, 0.0f), 3.0f)) << (2 * c);
    redo |= uint32_t(fabsf(__fsub_rn(q, r)) > 0.5f - 0x1p-18f) << c;
  }
  // the rare channels whose code the correctly rounded division decides
#pragma unroll 1
  for (; redo; redo &= redo - 1) {
    const int c = __ffs(redo) - 1;
    const uint32_t w = c < 4 ? (c < 2 ? vu[0] : vu[1]) : (c < 6 ? vu[2] : vu[3]);
    const uint32_t q = group_code(__uint_as_float(c & 1 ? w & 0xffff0000u : w << 16), gp);
    bits = (bits & ~(3u << (2 * c))) | (q << (2 * c));
  }
  if (gp.s == 0.0f) bits = 0;
  return gp;
}

}  // namespace kv2
