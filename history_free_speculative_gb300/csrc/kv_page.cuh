// The paged 4-bit cache's record of one (page, KV head): layout and conversions.
#pragma once

#include <cuda_fp16.h>

#include "internal.h"

namespace dlite {
namespace kv {

constexpr int kPage = DLITE_KV_PAGE;

// Byte offsets inside a record of 72 d_h bytes.
__host__ __device__ constexpr int rec_bytes(int d_h) { return 72 * d_h; }
__host__ __device__ constexpr int v_off(int d_h) { return 32 * d_h; }
__host__ __device__ constexpr int ks_off(int d_h) { return 64 * d_h; }
__host__ __device__ constexpr int vs_off(int d_h) { return 68 * d_h; }

// Two e2m1 codes (a byte, low nibble first) / two e4m3 numbers as an f16 pair. Both are
// exact, and so is the product of a code and a scale (2 + 4 significant bits, 2^-10..2688).
// byte B of a word of codes
template <int B>
__device__ __forceinline__ uint32_t fp4x2_of(uint32_t w) {
  uint32_t r;
  if constexpr (B == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (B == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (B == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t fp8x2_to_f16x2(uint16_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(two));
  return r;
}
// Nearest e4m3 of s (0 <= s <= 448), as a byte, and its value.
__device__ __forceinline__ uint32_t f32_to_fp8(float s) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(s));
  return r & 0xffu;
}
__device__ __forceinline__ float fp8_to_f32(uint32_t byte) {
  const uint32_t h = fp8x2_to_f16x2((uint16_t)byte);
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}
// Nearest e2m1 codes of 8 numbers, ties to even, saturating: nibble e is v[e]'s.
__device__ __forceinline__ uint32_t f32x8_to_fp4(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Codes (nibble e of the pair lo, hi: column e) and scale byte of 16 columns.
// v is overwritten. Returns whether a value was NaN or infinite.
//
// A code is the nearest to the fp32 quotient v / s. It is had without 16 divisions: with r the rounded 1 / s and q = v r, one
// correction q + (v - q s) r, whose residual is exact (s has four significant bits), is v / s to 2^-46 before its rounding. The
// borders t between codes (1/4, 3/4 .. 5) are fp32 numbers and so are the t s: at v = t s the sum rounds to t, the tie that the
// quotient is, and the next fp32 number after t s is more than half a step of t away from t after the division (2^-23 / m
// of t, m < 2 the significand of t s, against 2^-24 over that of t), so both fall on the same side. Overflow: v / s is below 7 unless s is
// the largest scale, 448. The sign is v's: a zero keeps it.
__device__ __forceinline__ bool quantise16(float (&v)[16], float inv_exp, uint2& codes, uint32_t& scale) {
  float amax = 0.f, odd = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] *= inv_exp;
    amax = fmaxf(amax, fabsf(v[i]));
    odd = fmaf(v[i], 0.f, odd);  // a NaN once a value is not finite
  }
  const bool bad = odd != 0.f;
  if (bad) {
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (fabsf(v[i]) <= 3.402823466e38f) amax = fmaxf(amax, fabsf(v[i]));
    const float far = fminf(2.f * amax, 3.402823466e38f);  // over 6 s, and its quotient is finite
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(fabsf(v[i]) <= 3.402823466e38f)) v[i] = v[i] != v[i] ? 0.f : copysignf(far, v[i]);
  }
  scale = f32_to_fp8(fminf(__fdiv_rn(amax, 6.f), 448.f));
  const float s = fp8_to_f32(scale);
  const float r = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = v[8 * i + e], q0 = x * r;
      q[e] = copysignf(fmaf(fmaf(-q0, s, x), r, q0), x);
    }
    w[i] = s > 0.f ? f32x8_to_fp4(q) : 0u;
  }
  codes = make_uint2(w[0], w[1]);
  return bad;
}

// Host checks shared by the cache's calls.
inline int check_cache(const dlite_kv_cache& c, int B, int T, const int64_t* pos, const int32_t* n_rows, const int* status) {
  if (!c.pages || !c.block_table || !pos) return DLITE_ERR_INVALID_ARG;
  if (((uintptr_t)c.pages & 15) || ((uintptr_t)pos & 7) || !aligned4(c.block_table, n_rows, status)) return DLITE_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || c.n_pages < 1 || c.n_kv < 1 || c.max_pages < 1) return DLITE_ERR_INVALID_ARG;
  if (c.k_exp < -64 || c.k_exp > 64 || c.v_exp < -64 || c.v_exp > 64) return DLITE_ERR_INVALID_ARG;
  if ((c.d_h != 64 && c.d_h != 128) || c.n_kv > 32767 || B > 65535 || c.max_pages >= (1 << 25) || T >= (1 << 30))
    return DLITE_ERR_UNSUPPORTED_SHAPE;
  return DLITE_OK;
}

}  // namespace kv
}  // namespace dlite
