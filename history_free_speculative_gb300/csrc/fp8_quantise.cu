// Activations and weights into 8 bits with a scale per block.
//
// Rows: optionally total = x + residual (rounded to the stream's type and stored), then y = total / sqrt(mean total^2 + eps) gain, then the
// codes of y. A thread holds 16 neighbouring columns, so eight neighbouring threads hold a block and its maximum is three shuffles (with eight columns a
// thread the norm kernel was bound by its issue slots, 300 instructions a warp and row).
// With a norm a CTA takes whole rows (the sum of squares is over the row); without one the
// row's pieces go to CTAs of their own.
#include <algorithm>
#include <type_traits>

#include "fp8.cuh"
#include "row_ring.cuh"

namespace dlite {
namespace {

using fp8::kBlock;

constexpr int kPer = 16;  // columns of a thread

struct QuantiseArgs {
  int rows, T, K;
  const void* x;
  long long xs;
  const void* res;
  long long rs;
  void* total;
  long long ts;
  const void* gain;
  float eps, inv_k;  // inv_k = 1 / K
  uint8_t* codes;
  long long cs;
  float* scale;
  const int32_t* n_rows;
  int* status;
};

// Columns [c, c + 16) of a row as they are stored, zeros past K
template <typename T>
struct Piece {
  T e[kPer];
  __device__ __forceinline__ void to(float (&v)[kPer]) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = to_f32(e[i]);
  }
};
// Rows off 16 bytes (VEC false): the whole warp takes its 512 columns side by side, through shared memory of its own. Column by column, a lane's
// accesses 32 or 64 bytes apart, 8,192 rows of 4,095 with norm and residual took 221 us (bf16) and 312 (float32), so 72 and 85; 16 rows of 1,335 3.4
// and 3.6.
constexpr int kWarpCols = 32 * kPer;
// Column j's place in it: float32 columns' 16-byte pieces in an order in which eight lanes' reads of theirs meet in no bank (8,192 rows of 4,095 with
// norm and residual 126 -> 90 us). 16-bit ones as they come: two lanes meet, and the other order cost more in addresses (72 -> 81).
template <typename T>
__device__ __forceinline__ int place(int j) {
  return sizeof(T) == 4 ? j ^ (j >> 5 & 3) << 2 : j;
}
template <typename T>
__device__ __forceinline__ void warp_columns(const T* row, T* buf, int c0, int K) {  // buf[place(i)] = row[c0 + i], zeros past K
  const int lane = threadIdx.x & 31;
  if (sizeof(T) == 2 && ((uintptr_t)(row + c0) & 3) == 0) {
    uint32_t w[kPer / 2];  // all loads before the first store, which they might name
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
      const int j = 2 * (lane + 32 * i);
      w[i] = 0;
      if (c0 + j + 1 < K)
        w[i] = *reinterpret_cast<const uint32_t*>(row + c0 + j);
      else if (c0 + j < K)
        w[i] = *reinterpret_cast<const uint16_t*>(row + c0 + j);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) *reinterpret_cast<uint32_t*>(buf + place<T>(2 * (lane + 32 * i))) = w[i];
  } else {
    T w[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) w[i] = c0 + lane + 32 * i < K ? row[c0 + lane + 32 * i] : T(0.f);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kPer; ++i) buf[place<T>(lane + 32 * i)] = w[i];
  }
  __syncwarp();
}
template <typename T, bool VEC>
__device__ __forceinline__ Piece<T> load_piece(const T* row, int c, int K, T* buf) {
  constexpr int E = 16 / sizeof(T);
  Piece<T> r;
  if (VEC) {  // K is a multiple of 8 here
#pragma unroll
    for (int i = 0; i < kPer / E; ++i)
      reinterpret_cast<uint4*>(r.e)[i] = c + i * E < K ? reinterpret_cast<const uint4*>(row + c)[i] : make_uint4(0, 0, 0, 0);
  } else {
    const int lane = threadIdx.x & 31;
    warp_columns(row, buf, c - lane * kPer, K);
#pragma unroll
    for (int i = 0; i < kPer / E; ++i) reinterpret_cast<uint4*>(r.e)[i] = *reinterpret_cast<const uint4*>(buf + place<T>(lane * kPer + i * E));
  }
  return r;
}
__device__ __forceinline__ float rounded(float v, float*) { return v; }
__device__ __forceinline__ float rounded(float v, bf16*) { return round_bf16(v); }
template <typename T, bool VEC>
__device__ __forceinline__ void store_piece(T* row, int c, int K, const float (&v)[kPer], T* buf) {
  constexpr int E = 16 / sizeof(T);
  Piece<T> r;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if constexpr (sizeof(T) == 2)
      r.e[i] = __float2bfloat16_rn(v[i]);
    else
      r.e[i] = v[i];
  }
  if (VEC) {
#pragma unroll
    for (int i = 0; i < kPer / E; ++i)
      if (c + i * E < K) reinterpret_cast<uint4*>(row + c)[i] = reinterpret_cast<const uint4*>(r.e)[i];
  } else {
    const int lane = threadIdx.x & 31, c0 = c - lane * kPer;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kPer / E; ++i) *reinterpret_cast<uint4*>(buf + place<T>(lane * kPer + i * E)) = reinterpret_cast<const uint4*>(r.e)[i];
    __syncwarp();
    if (sizeof(T) == 2 && ((uintptr_t)(row + c0) & 3) == 0) {
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) {
        const int j = 2 * (lane + 32 * i);
        if (c0 + j + 1 < K)
          *reinterpret_cast<uint32_t*>(row + c0 + j) = *reinterpret_cast<const uint32_t*>(buf + place<T>(j));
        else if (c0 + j < K)
          row[c0 + j] = buf[place<T>(j)];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (c0 + lane + 32 * i < K) row[c0 + lane + 32 * i] = buf[place<T>(lane + 32 * i)];
    }
  }
}

// Codes and scale of the eight threads' block; c is this thread's first column.
__device__ __forceinline__ void quantise_piece(const QuantiseArgs& a, int row, int c, float (&v)[kPer], bool& bad) {
  float amax = fp8::finite_max(v, bad);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int e = fp8::block_exponent(amax);
  const float inv = fp8::exp2i(-e);
  if (c >= a.K) return;
  uint32_t w[kPer / 4];
#pragma unroll
  for (int i = 0; i < kPer / 4; ++i) w[i] = fp8::codes4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
  uint8_t* dst = a.codes + (long long)row * a.cs + c;
  if (c + kPer <= a.K) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (c + i < a.K) dst[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
  if (c % kBlock == 0) a.scale[(long long)(c / kBlock) * a.rows + row] = fp8::exp2i(e);
}

// v = x + residual in the stream's type
template <typename T>
__device__ __forceinline__ void add_residual(const Piece<T>& res, float (&v)[kPer]) {
  float r[kPer];
  res.to(r);
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = rounded(v[i] + r[i], (T*)nullptr);
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_total(const QuantiseArgs& a, int row, int c, const float (&v)[kPer], T* buf) {
  store_piece<T, VEC>(static_cast<T*>(a.total) + row * a.ts, c, a.K, v, buf);
}

// Without a norm: CTA (row, piece of the row).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) fp8_quantise_kernel(const QuantiseArgs a) {
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, c = (blockIdx.y * blockDim.x + threadIdx.x) * kPer;
  if (!fp8::valid_row(a.n_rows, a.T, row)) return;
  __shared__ __align__(16) T bufs[VEC ? 1 : 8][VEC ? 8 : kWarpCols];
  T* buf = bufs[VEC ? 0 : threadIdx.x >> 5];
  float v[kPer];
  const Piece<T> x = load_piece<T, VEC>(static_cast<const T*>(a.x) + row * a.xs, c, a.K, buf);
  if (a.res) {
    const Piece<T> r = load_piece<T, VEC>(static_cast<const T*>(a.res) + row * a.rs, c, a.K, buf);
    x.to(v);
    add_residual(r, v);
    store_total<T, VEC>(a, row, c, v, buf);
  } else {
    x.to(v);
  }
  bool bad = false;
  quantise_piece(a, row, c, v, bad);
  if (bad) flag_status(a.status, kDevNonfinite);
}

// The block's sum of v, in every thread, in an order of its own size alone. red: 32 floats that nobody else reads before the next barrier but one.
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : 0.f);
}

// With a norm, rows on 16 bytes of up to 16 x 1,024 columns: a CTA takes rows in turn out of a ring in shared memory that bulk copies fill a
// few rows ahead. What bounds it is the bytes on their way: 8,192 rows of 4,096 bf16 columns with the residual sum took 71 us with one row a
// CTA and 69 with the next row's loads in registers, 32 KB an SM on their way in both.
constexpr int kRing = 4;
template <typename T>
__global__ void __launch_bounds__(1024) fp8_norm_quantise_kernel(const QuantiseArgs a, const int slots) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[2][32];
  __shared__ uint64_t full[kRing];
  __shared__ int gave_up[2];
  const int c = threadIdx.x * kPer, bytes = a.K * (int)sizeof(T), slot_bytes = a.res ? 2 * bytes : bytes;
  if (threadIdx.x == 0) {
    for (int i = 0; i < slots; ++i) tc::mbar_init(tc::su32(full + i), 1);
    gave_up[0] = gave_up[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_trigger();
  pdl_wait();
  const Piece<T> gain = load_piece<T, true>(static_cast<const T*>(a.gain), c, a.K, nullptr);
  auto next_row = [&](int row) {
    while (row < a.rows && !fp8::valid_row(a.n_rows, a.T, row)) row += gridDim.x;
    return row;
  };
  auto copy = [&](int row, int slot) {  // thread 0
    const uint32_t dst = tc::su32(ring + (size_t)slot * slot_bytes), bar = tc::su32(full + slot);
    tc::mbar_expect_tx(bar, slot_bytes);
    tc::bulk_load(dst, static_cast<const T*>(a.x) + row * a.xs, bytes, bar);
    if (a.res) tc::bulk_load(dst + bytes, static_cast<const T*>(a.res) + row * a.rs, bytes, bar);
  };
  RowRing r = {tc::su32(full), slots, gave_up, a.status};
  int row = next_row(blockIdx.x), ahead = row;
  if (threadIdx.x == 0)
    for (; r.flying < slots && ahead < a.rows; ++r.flying, ahead = next_row(ahead + gridDim.x)) copy(ahead, r.flying);
  __syncthreads();  // the barriers are there
  bool bad = false;
  while (row < a.rows) {
    const bool there = r.wait();
    const T* at = reinterpret_cast<const T*>(ring + (size_t)r.slot * slot_bytes);
    float v[kPer], ss = 0.f;
    load_piece<T, true>(at, c, a.K, nullptr).to(v);
    if (a.res) {
      add_residual(load_piece<T, true>(at + a.K, c, a.K, nullptr), v);
      // ahead of the barrier: 8,192 rows of 12,288 take 118 us so, 130 with the stores behind it
      if (there) store_total<T, true>(a, row, c, v, nullptr);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) ss = fmaf(v[i], v[i], ss);
    const float inv = rsqrtf(fmaf(row_sum(ss, red[r.parity]), a.inv_k, a.eps));
    if (r.late()) break;  // a slot that was not filled holds anything
    if (threadIdx.x == 0) {  // the sum's barrier: the slot is read
      if (ahead < a.rows) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        copy(ahead, r.slot);
        ahead = next_row(ahead + gridDim.x);
      } else {
        r.used();
      }
    }
    float g[kPer];
    gain.to(g);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = v[i] * inv * g[i];
    quantise_piece(a, row, c, v, bad);
    r.next();
    row = next_row(row + gridDim.x);
  }
  if (threadIdx.x == 0) r.drain();
  if (bad) flag_status(a.status, kDevNonfinite);
}

// With a norm, other rows: a CTA takes a row and reads its columns twice.
template <typename T, bool VEC>
__global__ void __launch_bounds__(VEC ? 1024 : 512) fp8_norm_quantise_wide_kernel(const QuantiseArgs a) {
  __shared__ float red[32];
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, step = blockDim.x * kPer;
  if (!fp8::valid_row(a.n_rows, a.T, row)) return;
  const T* x = static_cast<const T*>(a.x) + row * a.xs;
  const T* total = static_cast<const T*>(a.total) + row * a.ts;
  __shared__ __align__(16) T bufs[VEC ? 1 : 16][VEC ? 8 : kWarpCols];
  T* buf = bufs[VEC ? 0 : threadIdx.x >> 5];
  float v[kPer], g[kPer], ss = 0.f;
  // whole warps walk together: they load together, and a block's maximum is taken by all lanes
  for (int c = threadIdx.x * kPer; c - (int)threadIdx.x * kPer < a.K; c += step) {
    load_piece<T, VEC>(x, c, a.K, buf).to(v);
    if (a.res) {
      add_residual(load_piece<T, VEC>(static_cast<const T*>(a.res) + row * a.rs, c, a.K, buf), v);
      store_total<T, VEC>(a, row, c, v, buf);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) ss = fmaf(v[i], v[i], ss);
  }
  const float inv = rsqrtf(fmaf(row_sum(ss, red), a.inv_k, a.eps));
  bool bad = false;
  for (int c = threadIdx.x * kPer; c - (int)threadIdx.x * kPer < a.K; c += step) {
    load_piece<T, VEC>(a.res ? total : x, c, a.K, buf).to(v);  // this warp's own stores
    load_piece<T, VEC>(static_cast<const T*>(a.gain), c, a.K, buf).to(g);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = v[i] * inv * g[i];
    quantise_piece(a, row, c, v, bad);
  }
  if (bad) flag_status(a.status, kDevNonfinite);
}

// A weight's block of 128 x 128: one CTA, 16 rows a warp, four columns a lane, read once and held in registers. Magnitudes compare as integers; a
// block that is not finite is found by its maximum and takes a second way. 151,936 x 4,096 took 305 us
// from bf16 and 446 from float32, 6.1 and 7.0 TB/s (580 and 565 with a test of each element, at two CTAs an SM): HBM bounds it.
// From bf16 rows off 16 bytes four CTAs an SM cost three registers spilled, and are the faster all the same: 151,936 x 4,095 356 us, 381 at three.
template <typename T>
using Word4 = typename std::conditional<sizeof(T) == 4, uint4, uint2>::type;
__device__ __forceinline__ uint32_t magnitudes(uint32_t m, uint4 w) {
  return max(max(max(m, w.x & 0x7fffffffu), w.y & 0x7fffffffu), max(w.z & 0x7fffffffu, w.w & 0x7fffffffu));
}
__device__ __forceinline__ uint32_t magnitudes(uint32_t m, uint2 w) { return __vmaxu2(__vmaxu2(m, w.x & 0x7fff7fffu), w.y & 0x7fff7fffu); }
__device__ __forceinline__ void floats4(uint4 w, float (&v)[4]) {
  v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void floats4(uint2 w, float (&v)[4]) {
  v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
  v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
}
// The block's maximum, in every thread. red: 8 words that nobody else reads or writes.
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* red) {
  m = __reduce_max_sync(~0u, m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, red[i]);
  return m;
}
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2)
    fp8_weight_kernel(const T* w, long long ws, int N, int K, uint8_t* codes, long long cs, float* scale, int* status) {
  __shared__ uint32_t red[2][8];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = blockIdx.x * kBlock + 4 * lane;
  Word4<T> held[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int n = blockIdx.y * kBlock + 8 * i + warp;
    const T* at = w + n * ws + k;
    held[i] = Word4<T>{};
    if (VEC) {  // K is a multiple of 4, rows on 16 bytes
      if (n < N && k < K) held[i] = *reinterpret_cast<const Word4<T>*>(at);
    } else {
      T e[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = n < N && k + j < K ? at[j] : T(0.f);
      memcpy(&held[i], e, sizeof(held[i]));
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = magnitudes(m, held[i]);
  if (sizeof(T) == 2) m = max(m >> 16, m & 0xffffu) << 16;
  m = block_max(m, red[0]);
  const bool bad = m >= 0x7f800000u;
  if (bad) {  // the largest finite one
    m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v[4];
      floats4(held[i], v);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (fabsf(v[j]) <= 3.402823466e38f) m = max(m, __float_as_uint(fabsf(v[j])));
    }
    m = block_max(m, red[1]);
  }
  const int e = fp8::block_exponent(__uint_as_float(m));
  const float inv = fp8::exp2i(-e);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int n = blockIdx.y * kBlock + 8 * i + warp;
    if (n >= N) break;
    float v[4];
    floats4(held[i], v);
    if (bad) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (!(fabsf(v[j]) <= 3.402823466e38f)) v[j] = __uint_as_float(0x7fffffffu);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= inv;
    const uint32_t c = fp8::codes4(v[0], v[1], v[2], v[3]);
    uint8_t* dst = codes + n * cs + k;
    if (k + 4 <= K) {
      *reinterpret_cast<uint32_t*>(dst) = c;
    } else {
      for (int j = 0; j < K - k; ++j) dst[j] = (uint8_t)(c >> (8 * j));
    }
  }
  if (threadIdx.x == 0) scale[(long long)blockIdx.y * gridDim.x + blockIdx.x] = fp8::exp2i(e);
  if (bad && threadIdx.x == 0) flag_status(status, kDevNonfinite);
}
template <typename T>
cudaError_t launch_weight(const dlite_fp8_weight_args& g, cudaStream_t s) {
  const dim3 grid(fp8::blocks_of(g.K), fp8::blocks_of(g.N));
  const bool vec = !((uintptr_t)g.w & 15) && g.K % 4 == 0 && g.w_stride % (16 / sizeof(T)) == 0;
  return launch_pdl(vec ? fp8_weight_kernel<T, true> : fp8_weight_kernel<T, false>, grid, dim3(256), 0, s, static_cast<const T*>(g.w),
                    (long long)g.w_stride, g.N, g.K, g.codes, (long long)g.codes_stride, g.scale, g.status);
}

template <typename T, bool VEC>
cudaError_t launch_quantise(const QuantiseArgs& a, cudaStream_t s) {
  const int threads = (a.K + kPer - 1) / kPer;
  if (!a.gain) {
    const int t = std::min(256, (threads + 31) / 32 * 32);
    return launch_pdl(fp8_quantise_kernel<T, VEC>, dim3(a.rows, (threads + t - 1) / t), dim3(t), 0, s, a);
  }
  const int t = std::min(1024, (threads + 31) / 32 * 32), row_bytes = a.K * (int)sizeof(T) * (a.res ? 2 : 1);
  if constexpr (VEC) {
    // few rows: nothing to fetch ahead (600 rows of 4,096: 4.8 us read twice, 5.3 over the ring; 1,024: 8.4 both; 8,192: 40)
    if (threads <= t && a.rows > 4 * device_sms()) {
      constexpr int kMost = 200 * 1024;
      const int ctas = std::min(16, std::max(1, 1536 / t)), slots = std::max(1, std::min(kRing, kMost / ctas / row_bytes));
      cudaError_t e = cudaFuncSetAttribute(fp8_norm_quantise_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
      if (e != cudaSuccess) return e;
      return launch_pdl(fp8_norm_quantise_kernel<T>, dim3(std::min(a.rows, device_sms() * ctas)), dim3(t), (size_t)slots * row_bytes, s, a, slots);
    }
  }
  return launch_pdl(fp8_norm_quantise_wide_kernel<T, VEC>, dim3(a.rows), dim3(VEC ? t : std::min(t, 512)), 0, s, a);
}

}  // namespace
}  // namespace dlite

extern "C" int dlite_fp8_quantise(const dlite_fp8_quantise_args* g, dlite_stream_t stream) {
  using namespace dlite;
  if (!g || !g->x || !g->codes || !g->scale || (g->residual != nullptr) != (g->total != nullptr)) return DLITE_ERR_INVALID_ARG;
  if (g->B < 1 || g->T < 1 || g->K < 1 || (g->dtype != DLITE_F32 && g->dtype != DLITE_BF16)) return DLITE_ERR_INVALID_ARG;
  if (g->gain && !(g->eps >= 0.f && g->eps <= 3.402823466e38f)) return DLITE_ERR_INVALID_ARG;
  const int es = g->dtype == DLITE_F32 ? 4 : 2, V = 16 / es;
  if (((uintptr_t)g->x | (uintptr_t)g->residual | (uintptr_t)g->total | (uintptr_t)g->gain) % es || !aligned4(g->scale, g->n_rows, g->status) ||
      ((uintptr_t)g->codes & 15))
    return DLITE_ERR_INVALID_ARG;
  if (g->x_stride < g->K || g->codes_stride < g->K || g->codes_stride % 16) return DLITE_ERR_INVALID_ARG;
  if (g->residual && (g->residual_stride < g->K || g->total_stride < g->K)) return DLITE_ERR_INVALID_ARG;
  if ((g->total == g->residual && g->total_stride != g->residual_stride) || (g->total == g->x && g->total_stride != g->x_stride))
    return DLITE_ERR_INVALID_ARG;
  if ((long long)g->B * g->T > DLITE_FP8_MAX_ROWS || g->K > DLITE_FP8_MAX_K) return DLITE_ERR_UNSUPPORTED_SHAPE;
  QuantiseArgs a = {};
  a.rows = g->B * g->T;
  a.T = g->T;
  a.K = g->K;
  a.x = g->x;
  a.xs = g->x_stride;
  a.res = g->residual;
  a.rs = g->residual_stride;
  a.total = g->total;
  a.ts = g->total_stride;
  a.gain = g->gain;
  a.eps = g->eps;
  a.inv_k = 1.f / (float)g->K;
  a.codes = g->codes;
  a.cs = g->codes_stride;
  a.scale = g->scale;
  a.n_rows = g->n_rows;
  a.status = g->status;
  const Rows x = {g->x, a.rows, a.xs * es, (long long)a.K * es}, res = {g->residual, a.rows, a.rs * es, x.width},
             total = {g->total, a.rows, a.ts * es, x.width}, gain = {g->gain, 1, 0, x.width}, codes = {g->codes, a.rows, a.cs, a.K},
             scale = {g->scale, 1, 0, 4LL * a.rows * fp8::blocks_of(a.K)};
  if (!apart_of(codes, x, res, total, gain, scale) || !apart_of(scale, x, res, total, gain) || !apart(total, gain) ||
      (total.at != x.at && !apart(total, x)) || (total.at != res.at && !apart(total, res)))
    return DLITE_ERR_INVALID_ARG;
  const bool vec = !(((uintptr_t)g->x | (uintptr_t)g->residual | (uintptr_t)g->total | (uintptr_t)g->gain) & 15) && g->K % 8 == 0 &&
                   g->x_stride % V == 0 && (!g->residual || (g->residual_stride % V == 0 && g->total_stride % V == 0));
  const cudaStream_t s = (cudaStream_t)stream;
  if (g->dtype == DLITE_F32)
    return launch_status(vec ? launch_quantise<float, true>(a, s) : launch_quantise<float, false>(a, s));
  return launch_status(vec ? launch_quantise<bf16, true>(a, s) : launch_quantise<bf16, false>(a, s));
}

extern "C" int dlite_fp8_weight(const dlite_fp8_weight_args* g, dlite_stream_t stream) {
  using namespace dlite;
  if (!g || !g->w || !g->codes || !g->scale || g->N < 1 || g->K < 1) return DLITE_ERR_INVALID_ARG;
  if (g->dtype != DLITE_F32 && g->dtype != DLITE_BF16) return DLITE_ERR_INVALID_ARG;
  if ((uintptr_t)g->w % (g->dtype == DLITE_F32 ? 4 : 2) || !aligned4(g->scale, g->status) || ((uintptr_t)g->codes & 15)) return DLITE_ERR_INVALID_ARG;
  if (g->w_stride < g->K || g->codes_stride < g->K || g->codes_stride % 16) return DLITE_ERR_INVALID_ARG;
  if (g->K > DLITE_FP8_MAX_K || g->N > DLITE_FP8_MAX_N) return DLITE_ERR_UNSUPPORTED_SHAPE;
  const int es = g->dtype == DLITE_F32 ? 4 : 2;
  const Rows w = {g->w, g->N, g->w_stride * es, (long long)g->K * es}, codes = {g->codes, g->N, g->codes_stride, g->K},
             scale = {g->scale, 1, 0, 4LL * fp8::blocks_of(g->N) * fp8::blocks_of(g->K)};
  if (!apart_of(codes, w, scale) || !apart(scale, w)) return DLITE_ERR_INVALID_ARG;
  const cudaStream_t s = (cudaStream_t)stream;
  return launch_status(g->dtype == DLITE_F32 ? launch_weight<float>(*g, s) : launch_weight<bf16>(*g, s));
}
