// e4m3 values with one fp32 scale for a block of 128: the arithmetic that the
// quantiser and the SwiGLU epilogue share.
#pragma once

#include "common.h"

namespace moe {

constexpr float kE4m3Max = 448.0f;
// the magnitude a block is scaled by is at least this, so that neither the
// scale nor its reciprocal leaves fp32's normal range
constexpr float kQuantTiny = 7.888609052210118e-31f;  // 2^-100

// Quotients 448 x / amax of one block: 7/8 x by amax, times 512, by one Newton
// step on the hardware reciprocal, within 2^-23 of the real quotient and equal
// to it where it is an fp32 number (the step's remainder is then exact).  7/8 x
// is exact for bf16 x, so a quotient that lies half way between two e4m3
// values is met exactly and rounds to even, and no other comes that near one;
// a product with a rounded 448 / amax would move it off the tie.  Of fp32 x
// 7/8 x is rounded too: quotients within 2^-22 of a tie may take either
// neighbour.  amax above 1 is brought
// down by 2^-64 first (exact), so its reciprocal is a normal number.
struct BlockQuant {
  float c, d, r;
  __device__ __forceinline__ explicit BlockQuant(float amax) {
    const float pre = amax > 1.0f ? 5.421010862427522e-20f : 1.0f;  // 2^-64
    c = 0.875f * pre;
    d = amax * pre;
    r = __builtin_amdgcn_rcpf(d);
  }
  // |result| <= 448 for |x| <= amax
  __device__ __forceinline__ float operator()(float x) const {
    const float y = x * c;
    const float q = y * r;
    return fmaf(fmaf(-q, d, y), r, q) * 512.0f;
  }
};

__device__ __forceinline__ float block_scale(float amax) { return amax / kE4m3Max; }

// Four values to four e4m3 bytes (round to nearest even).
__device__ __forceinline__ uint32_t e4m3_quad(float a, float b, float c, float d) {
  int p = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  p = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, p, true);
  return static_cast<uint32_t>(p);
}

}  // namespace moe
