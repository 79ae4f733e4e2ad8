// Shared parts of the 8-bit products: the block format, arguments, tensor maps' boxes.
//
// Activations: e4m3 codes and one scale per (row, 128 columns), the least 2^e (e >= -126) with max |x| <= 448 2^e. A power of two makes
// the code one rounding of an exact product, whatever computes it, and costs e4m3 no precision: its steps are relative down to 2^-6.
// Weights: e4m3 codes and a float32 scale per 128 x 128 elements.
#pragma once

#include <cuda.h>

#include "tc_device.cuh"

namespace dlite {
namespace fp8 {

constexpr int kBlock = DLITE_FP8_BLOCK;
static_assert(kBlock == 128, "a k block is one 128-byte swizzled row of the operand tiles");

__host__ __device__ constexpr int blocks_of(int n) { return n / kBlock + (n % kBlock != 0); }

// Exponent of a block's scale: amax = m 2^k, 448 = 1.75 2^8, so that e = k - 8, or k - 7 where the significand is above 1.75 (the
// addition carries into the exponent there).
__device__ __forceinline__ int block_exponent(float amax) {
  return max((int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 135, -126);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }  // -126 <= e <= 127

// Codes of four numbers (first lowest): nearest, ties to even. NaN becomes NaN.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// The largest finite |v| of N numbers; what is not finite becomes NaN (the format holds no infinity) and sets `bad`.
template <int N>
__device__ __forceinline__ float finite_max(float (&v)[N], bool& bad) {
  float amax = 0.f, odd = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    amax = fmaxf(amax, fabsf(v[i]));
    odd = fmaf(v[i], 0.f, odd);  // NaN once a number is not finite
  }
  if (odd != 0.f) {
    bad = true;
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (fabsf(v[i]) <= 3.402823466e38f)
        amax = fmaxf(amax, fabsf(v[i]));
      else
        v[i] = __uint_as_float(0x7fffffffu);
    }
  }
  return amax;
}

// A row's place among the requests' blocks: row (b, t) is valid iff t < n_rows[b].
__device__ __forceinline__ bool valid_row(const int32_t* n_rows, int T, int row) {
  return !n_rows || row % T < n_rows[row / T];
}

// Instruction descriptor, kind::f8f6f4: float32 sums, e4m3 on both sides, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void umma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The gated activation g / (1 + exp(-g)) u, of two pairs of sums at once. exp2 within 2^-22, its argument's rounding |g| 2^-23, the reciprocal within
// 2^-23: far below the 2^-4 of the code that it becomes. (With expf and a division the 16,384 results of a tile cost the many-row kernel 4 us.)
// As 1/4 over (1 + exp(-g)) / 4: the reciprocal instruction takes what is below 2^-126 to 0, where exp(-g) is still a float32
// number (g from -88.72 to -87.34); of the quarter it is above that. Past them exp(-g) is infinite and the result 0, as in float32.
__device__ __forceinline__ uint64_t gated2(uint64_t g, uint64_t u) {
  const uint64_t quarter = pack2f(0.25f, 0.25f), t = fma2(g, pack2f(-tc::kLog2e, -tc::kLog2e), pack2f(-2.f, -2.f));
  const uint64_t d = add2(quarter, pack2f(tc::ex2_approx(lo2f(t)), tc::ex2_approx(hi2f(t))));
  return mul2(mul2(g, mul2(quarter, pack2f(rcp_approx(lo2f(d)), rcp_approx(hi2f(d))))), u);
}

// One lane of a converged warp. Copies and products take their operands from uniform registers; in a branch on the lane's
// number each of them took 100 clocks to issue.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}
// Whether a phase is over, without waiting for it.
__device__ __forceinline__ bool mbar_peek(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// 32 columns of tensor memory, not waited for.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}
// Wait of a whole warp for an accumulator: every lane polls for itself (no vote in the polls), one vote at the end.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, int* status) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, status));
}
// A box of the map into L2, without waiting for the kernel before: the weights' way from HBM begins while that one still runs.
// (L2 is where all SMs' accesses meet: what the kernel before writes there afterwards is what the copy reads.)
__device__ __forceinline__ void prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y) : "memory");
}

struct ProductArgs {
  int rows, T;            // rows = B T
  int K, kblocks;
  int N;                  // outputs (gated: columns of the activation)
  const int32_t* n_rows;
  const float* xs;        // [kblocks][rows]: a warp, lane = row, reads a block's scales side by side
  const float* ws[2];     // [N / 128][kblocks]; gated: gate, up
  void* out;              // linear
  long long os;
  uint8_t* codes;         // gated
  long long cs;
  float* scale;           // [N / 128][rows]
  int vec;                // linear: rows of out on 16 bytes
  int* status;
};

// The products' operands in memory and their tensor maps: byte rows of K columns for boxes of 128 bytes under the 128-byte swizzle; columns and
// rows past a matrix read as 0.
struct Operands {
  const void* x;
  long long xs;
  const void* w[2];
  long long ws[2];
};
struct Maps {
  CUtensorMap x, w0, w1;
};
// To be called after a call of the runtime that needs the device's context (a kernel's attribute): in a host thread that has made no CUDA call
// yet the context is not current, and the encoder refuses.
bool make_maps(Maps& m, const Operands& o, const ProductArgs& p, int x_box, int w_box);

// The kernel for many rows (fp8_pair.cu): boxes of 128 rows of x, 128 (linear) or 64 (gated) weight rows.
double pairs_us(const ProductArgs& p, bool gated);  // an estimate of its time
cudaError_t launch_pairs(const Operands& o, const ProductArgs& p, bool gated, bool f32, cudaStream_t s);

}  // namespace fp8
}  // namespace dlite
