// The rotation of one pair of columns, shared by the rotary call and the cache
// append. Each product is rounded to fp32 before the sum (no fused multiply-add):
// the 4-bit codes of a rotated key are then the same on every path that
// follows this order, down to the bit.
#pragma once

#include "common.cuh"

namespace dlite {

__device__ __forceinline__ void rope_pair(float x0, float x1, float2 cs, float& y0, float& y1) {
  y0 = __fsub_rn(__fmul_rn(x0, cs.x), __fmul_rn(x1, cs.y));
  y1 = __fadd_rn(__fmul_rn(x1, cs.x), __fmul_rn(x0, cs.y));
}

}  // namespace dlite
