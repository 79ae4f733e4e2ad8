// The block-scaled products (fp8_linear.cu) for many rows: CTA pairs, 2-SM MMAs.
//
// A cluster of two CTAs walks tiles of 256 rows x 256 weight rows. Per k block of 128 columns four tcgen05.mma.cta_group::2
// kind::f8f6f4 (M = 256, N = 256, K = 32) write one of two accumulators in tensor memory (all its 512 columns); CTA c holds rows 128 c .. of x
// and rows 128 c .. of the weights in its shared memory and gets its 128 rows over all 256 columns. Eight epilogue warps a CTA take an
// accumulator times the block's scales into float32 sums in registers (lane = row, 128 columns a thread) while the
// tensor cores work on the next.
// What bounds it: the way round of an accumulator (products 512 clocks, commit to both CTAs, reads, hand-over to the CTA that issues), 1,600 to
// 1,800 clocks for two blocks, and under load the power cap (1,350 W). 8,192 rows over and over, with the clock that held: 6,144 x 4,096 168 to 171 us
// at 1.87 to 1.92 GHz (2.4 PFLOP/s), 4,096 x 12,288 345 to 349 us at 1.53 GHz (2.4), gated 12,288 x 4,096 630 to 658 us at 1.67 to 1.81 GHz (2.5 to 2.6);
// six calls behind a pause 169 to 185, 306 to 317 and 594 to 602 us. Without the reads, the hand-overs kept, the last two take 298 us at 2.06 GHz
// and 624 at 1.97; with the weights copied five times alone besides, 288 and 588: at full clock about 900 clocks a block stay, the hand-over's.
// Tried: 128 weight rows a step and four accumulators (371 us for 4,096 x 12,288: twice the waits); one-CTA products of 128 x 256 handed over
// inside the SM (309 us: an SM then takes in 48 KB a block where its way from L2 brings 64 bytes a clock); splits of the k blocks over clusters of
// four to eight CTAs for few tiles (few such clusters of whole-SM CTAs are resident at once).
// Gated: the 256 weight rows are [64 gate | 64 up] twice, so a thread holds 64 gate and 64 up columns of its row, and the two warps of a
// row exchange one maximum for the scale of its 128 results.
// Tiles go to the pairs row tiles first: the weights are read from HBM once, x stays in L2.
#include <algorithm>

#include "fp8.cuh"

namespace dlite {
namespace {

using fp8::kBlock;
using fp8::ProductArgs;

constexpr int kThreads = 128 + 256;           // copy warp, MMA warp, two that only make up the warpgroup; eight epilogue warps
// Registers a thread: the epilogue's sums (128) and two loads of 32 columns in flight need more than the launch's 168.
// 128 x 56 + 256 x 224 = 384 x 168, what the CTA was launched with.
constexpr int kRegsFew = 56, kRegsMany = 224;
constexpr int kStages = 5;
constexpr uint32_t kTile = 128 * 128;         // 128 rows of one k block
constexpr uint32_t kStage = 2 * kTile;        // this CTA's rows of x and of the weights
constexpr int kPitch = 144;                   // bytes of a staged row: 128 and 16 that take its chunks to other banks
constexpr uint32_t kStaging = 8 * 32 * kPitch;
// A thread's own scales of the blocks to come go to shared memory a few blocks ahead of their use, without registers or barriers: the
// thread that copies is the one that reads. (A load one block ahead was late wherever it missed the first cache: 8,192 rows of 4,096 x
// 12,288 took 404 us so, 290 with the copies.)
constexpr int kScalesAhead = 6, kScaleSlots = 8;
constexpr uint32_t kSmem = 1024 + 1024 + kStages * kStage + kStaging + kScaleSlots * 1024;
static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");

__device__ __forceinline__ void umma_e4m3_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}

__device__ __forceinline__ void copy_scale(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ float own_scale(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

constexpr int kMaxRowTiles = DLITE_FP8_MAX_ROWS / 256;

// Whether one of the 256 rows from row0 on is valid.
__device__ __forceinline__ bool live_tile(const ProductArgs& p, int row0) {
  const int end = min(row0 + 256, p.rows);
  for (int r = row0; r < end;) {
    const int b = r / p.T, t = r - b * p.T;
    if (t < p.n_rows[b]) return true;
    r += p.T - t;
  }
  return false;
}

// 32 staged rows of 128 bytes to rows off 16 bytes, lanes side by side, `cols` columns at most. 16 bytes a lane element by element, 770 rows of 260
// and 26,226 bf16 columns took 110 us, side by side 40 (26,224 on 16 bytes: 23); 4,096 of 4,096 and 4,099 116 and 75. In a kernel of its own: with
// both stores in one, rows on 16 bytes took 3 % more. (The few-row kernel keeps its scalar stores: 64 rows of 4,096 and 4,099 lose 0.25 us of 8.6 to
// them, and lanes side by side there cost its other calls 0.1 to 0.9 us.)
template <typename OUT>
__device__ __noinline__ void store_rows(OUT* dst, long long stride, const uint8_t* staged, uint32_t valid_rows, int cols) {
  constexpr int E = 4 / sizeof(OUT), kBatch = 8;
  const int lane = threadIdx.x & 31, c = lane * E;
  // 16 bits: a row on 4 bytes takes a lane's columns c and c + 1 as a word, any other row columns c + 1 and c + 2 and its first column alone
  const bool word0 = c + E <= cols, half0 = c + 1 == cols, word1 = lane < 31 && c + 2 < cols, half1 = !word1 && c + 1 < cols,
             first1 = lane == 0 && cols > 0;
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += kBatch) {
    uint32_t w[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) w[i] = reinterpret_cast<const uint32_t*>(staged + (r0 + i) * kPitch)[lane];
#pragma unroll
    for (int i = 0; i < kBatch; ++i, dst += stride) {
      const bool valid = valid_rows >> (r0 + i) & 1;
      if constexpr (E == 1) {
        if (valid && word0) dst[c] = __uint_as_float(w[i]);
      } else {
        uint16_t* d = reinterpret_cast<uint16_t*>(dst) + c;
        if (((uintptr_t)dst & 3) == 0) {
          if (valid && word0) *reinterpret_cast<uint32_t*>(d) = w[i];
          if (valid && half0) d[0] = (uint16_t)w[i];
        } else {
          const uint32_t next = __shfl_down_sync(~0u, w[i], 1);
          if (valid && word1) *reinterpret_cast<uint32_t*>(d + 1) = w[i] >> 16 | next << 16;
          if (valid && half1) d[1] = (uint16_t)(w[i] >> 16);
          if (valid && first1) d[0] = (uint16_t)w[i];
        }
      }
    }
  }
}

template <bool GATED, typename OUT, bool VEC>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw0, const __grid_constant__ CUtensorMap mw1,
                    const ProductArgs p, const int row_tiles, const int tiles) {
  // Shared memory: [barriers | pad to 1 KB] [stage 0] .. [epilogue staging] [scales]; stage = [x tile][weight tile]
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = (uint64_t*)base;
  const uint32_t full0 = tc::su32(bars), empty0 = full0 + 8 * kStages, accf0 = empty0 + 8 * kStages, acce0 = accf0 + 16, done = acce0 + 16;
  uint32_t* tmem_holder = (uint32_t*)(bars + 2 * kStages + 5);
  uint8_t* smem = base + 1024;
  __shared__ float row_max[2][128];
  __shared__ uint32_t live[kMaxRowTiles / 32];  // row tiles with a valid row

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_rank();
  const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(full0 + 8 * s, 1);
      tc::mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(accf0 + 8 * b, 1);
      tc::mbar_init(acce0 + 8 * b, 16);  // every epilogue warp of both CTAs
    }
    tc::mbar_init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::su32(tmem_holder)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync_all();  // both CTAs' barriers exist before any copy, commit or arrival reaches them
  tc::fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_trigger();
  pdl_wait();
  if (p.n_rows) {
    for (int i = threadIdx.x; i < (row_tiles + 31) / 32 * 32; i += kThreads) {  // whole warps
      const uint32_t bits = __ballot_sync(0xffffffffu, i < row_tiles && live_tile(p, i * 256));
      if (lane == 0) live[i >> 5] = bits;
    }
    __syncthreads();
  }
  auto skip = [&](int t) { return p.n_rows && !(live[(t % row_tiles) >> 5] >> ((t % row_tiles) & 31) & 1); };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (warp == 0 && fp8::elect_one()) {  // ---------------- copies (both CTAs; every one signals rank 0's full barrier)
      const uint32_t full_leader = tc::map_to_rank(full0, 0);
      int s = 0, issued = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs) {
        const int row0 = (t % row_tiles) * 256, n0 = t / row_tiles;
        if (skip(t)) continue;
        for (int kb = 0; kb < p.kblocks; ++kb) {
          if (issued >= kStages) ok = tc::mbar_wait(empty0 + 8 * s, ph ^ 1u, p.status);
          if (!ok) break;
          const uint32_t st = tc::su32(smem + s * kStage), bar = full_leader + 8 * s;
          if (rank == 0) tc::mbar_expect_tx(full0 + 8 * s, 2 * kStage);
          if (GATED) {
            tc::tma_load_2d_pair(st + kTile, &mw0, bar, kb * kBlock, n0 * 128 + (int)rank * 64);
            tc::tma_load_2d_pair(st + kTile + kTile / 2, &mw1, bar, kb * kBlock, n0 * 128 + (int)rank * 64);
          } else {
            tc::tma_load_2d_pair(st + kTile, &mw0, bar, kb * kBlock, n0 * 256 + (int)rank * 128);
          }
          tc::tma_load_2d_pair(st, &mx, bar, kb * kBlock, row0 + (int)rank * 128);
          ++issued;
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok && rank == 0)  // the copies in flight end (bounded) before the pair's memory is given back
        for (int i = 0; i < kStages && i < issued; ++i) {
          if (s == 0) {
            s = kStages;
            ph ^= 1u;
          }
          --s;
          tc::mbar_wait(full0 + 8 * s, ph, p.status);
        }
    } else if (warp == 1 && rank == 0 && fp8::elect_one()) {  // ---------------- products
      constexpr uint32_t idesc = fp8::idesc_e4m3(256, 256);
      const uint64_t desc0 = tc::sw128_desc(tc::su32(smem));
      // The tensor pipe stands still from the last product of a block to the first of the next if this lane is late: the barriers of
      // the next block are looked at before the last product.
      int s = 0, i = 0;
      uint32_t ph = 0;
      bool ok = true, ready = false;
      for (int t = pair; t < tiles && ok; t += pairs) {
        if (skip(t)) continue;
        for (int kb = 0; kb < p.kblocks; ++kb, ++i) {
          const int b = i & 1;
          if (!ready) {
            ok = (i < 2 || tc::mbar_wait(acce0 + 8 * b, (uint32_t)((i >> 1) - 1) & 1u, p.status)) && tc::mbar_wait(full0 + 8 * s, ph, p.status);
            if (!ok) break;
          }
          tc::fence_after();
          const uint64_t a0 = desc0 + (uint64_t)(kStage >> 4) * s, b0 = a0 + (kTile >> 4);
          const uint32_t empty = empty0 + 8 * s;
#pragma unroll
          for (int kk = 0; kk < 3; ++kk) umma_e4m3_pair(tmem + 256 * b, a0 + 2 * kk, b0 + 2 * kk, idesc, kk > 0);
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
          ready = (i == 0 || fp8::mbar_peek(acce0 + 8 * (b ^ 1), (uint32_t)((i - 1) >> 1) & 1u)) && fp8::mbar_peek(full0 + 8 * s, ph);
          umma_e4m3_pair(tmem + 256 * b, a0 + 6, b0 + 6, idesc, 1);
          tc::umma_commit_pair(accf0 + 8 * b);
          tc::umma_commit_pair(empty);
        }
      }
      // every product issued has finished before the pair's memory goes
      tc::umma_commit_pair(done);
      tc::mbar_wait(done, 0, p.status);
    }
  } else {  // ---------------- sums: lane = row, 128 columns a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
    const int q = warp & 3, eg = (warp - 4) >> 2;
    const uint32_t acce_leader = tc::map_to_rank(acce0, 0);
    uint8_t* staged = smem + kStages * kStage + (warp - 4) * 32 * kPitch;
    const int nb = fp8::blocks_of(p.N);
    const uint32_t scales = tc::su32(smem + kStages * kStage + kStaging) + threadIdx.x * 4 - 512;  // this thread's word of slot 0
    int i = 0;
    for (int t = pair; t < tiles; t += pairs) {
      const int row0 = (t % row_tiles) * 256, n0 = t / row_tiles;
      if (skip(t)) continue;
      const int wrow0 = row0 + (int)rank * 128 + q * 32, row = wrow0 + lane;
      const float* xs = p.xs + min(row, p.rows - 1);
#pragma unroll
      for (int k = 0; k < kScalesAhead; ++k) {
        if (k < p.kblocks) copy_scale(scales + k * 1024, xs);
        xs += p.rows;
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      const int wb = GATED ? n0 : min(2 * n0 + eg, nb - 1);      // a block past the last has no columns to write
      const float* w0 = p.ws[0] + (long long)wb * p.kblocks;
      const float* w1 = GATED ? p.ws[1] + (long long)wb * p.kblocks : w0;
      uint64_t acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0;
      float w0_next = w0[0], w1_next = w1[0];
      bool ok = true;
      for (int kb = 0; kb < p.kblocks; ++kb, ++i) {
        const int b = i & 1;
        asm volatile("cp.async.wait_group %0;" ::"n"(kScalesAhead - 1) : "memory");
        const float x = own_scale(scales + kb % kScaleSlots * 1024), s0 = x * w0_next, s1 = GATED ? x * w1_next : s0;
        if (kb + kScalesAhead < p.kblocks) copy_scale(scales + (kb + kScalesAhead) % kScaleSlots * 1024, xs);
        xs += p.rows;
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (kb + 1 < p.kblocks) {
          w0_next = w0[kb + 1];
          if (GATED) w1_next = w1[kb + 1];
        }
        ok = fp8::wait_all(accf0 + 8 * b, (uint32_t)(i >> 1) & 1u, p.status);
        if (!ok) break;
        tc::fence_after();
        const uint32_t t0 = tmem + ((uint32_t)(q * 32) << 16) + 256 * b + 128 * eg;
        uint32_t v[2][32];
        fp8::tmem_ld32(t0, v[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tc::tmem_wait_ld();
          if (c < 3) {
            fp8::tmem_ld32(t0 + 32 * (c + 1), v[(c + 1) & 1]);
          } else {  // all read: the accumulator is the products' again
            tc::fence_before();
            __syncwarp();
            // what this hands over was read from tensor memory, which tcgen05.fence orders: a release of the generic memory, at
            // the cluster's scope, doubled the kernel's time
            if (lane == 0)
              asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(acce_leader + 8 * b) : "memory");
          }
          const float sc = c < 2 ? s0 : s1;
          const uint64_t sc2 = pack2f(sc, sc);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            acc[16 * c + j] = fma2(pack2f(__uint_as_float(v[c & 1][2 * j]), __uint_as_float(v[c & 1][2 * j + 1])), sc2, acc[16 * c + j]);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");  // where a wait gave up: no copy is left on its way
      // the sums leave through this warp's staging, so that neighbouring lanes store neighbouring columns
      if constexpr (GATED) {
        float a[64];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const uint64_t two = fp8::gated2(acc[j], acc[32 + j]);
          a[2 * j] = lo2f(two);
          a[2 * j + 1] = hi2f(two);
        }
        bool bad = false;
        float amax = fp8::finite_max(a, bad);
        row_max[eg][q * 32 + lane] = ok ? amax : -1.f;
        asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
        const float other = row_max[eg ^ 1][q * 32 + lane];
        asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");  // read before the next tile's is written
        if (!ok || other < 0.f) break;  // where one warp of a row gave up both leave, so that none waits for the other
        amax = fmaxf(amax, other);
        const int e = fp8::block_exponent(amax);
        const float inv = fp8::exp2i(-e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 w;
          w.x = fp8::codes4(a[16 * j] * inv, a[16 * j + 1] * inv, a[16 * j + 2] * inv, a[16 * j + 3] * inv);
          w.y = fp8::codes4(a[16 * j + 4] * inv, a[16 * j + 5] * inv, a[16 * j + 6] * inv, a[16 * j + 7] * inv);
          w.z = fp8::codes4(a[16 * j + 8] * inv, a[16 * j + 9] * inv, a[16 * j + 10] * inv, a[16 * j + 11] * inv);
          w.w = fp8::codes4(a[16 * j + 12] * inv, a[16 * j + 13] * inv, a[16 * j + 14] * inv, a[16 * j + 15] * inv);
          *reinterpret_cast<uint4*>(staged + lane * kPitch + 16 * j) = w;
        }
        __syncwarp();  // the lanes read each other's rows below
        const bool valid = row < p.rows && fp8::valid_row(p.n_rows, p.T, row);
        if (valid && bad) flag_status(p.status, kDevNonfinite);
        if (valid && eg == 0) p.scale[(long long)n0 * p.rows + row] = fp8::exp2i(e);
        const uint32_t valid_rows = __ballot_sync(0xffffffffu, valid);
        const int n = n0 * 128 + eg * 64 + (lane & 3) * 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 8 * j + (lane >> 2);
          const uint4 w = *reinterpret_cast<const uint4*>(staged + r * kPitch + 16 * (lane & 3));
          if (!(valid_rows >> r & 1)) continue;
          uint8_t* dst = p.codes + (long long)(wrow0 + r) * p.cs + n;
          if (n + 16 <= p.N) {
            *reinterpret_cast<uint4*>(dst) = w;
          } else {
            const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (n + k < p.N) dst[k] = (uint8_t)(word[k >> 2] >> (8 * (k & 3)));
          }
        }
        __syncwarp();
      } else {
        if (!ok) break;
        constexpr int C = 128 / sizeof(OUT), E = 16 / sizeof(OUT);  // columns of a staged piece, of a 16-byte chunk
        const uint32_t valid_rows = __ballot_sync(0xffffffffu, row < p.rows && fp8::valid_row(p.n_rows, p.T, row));
#pragma unroll
        for (int piece = 0; piece < 128 / C; ++piece) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint4 w;
            const int a0 = (piece * C + j * E) / 2;
            if constexpr (sizeof(OUT) == 2) {
              uint32_t h[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 two = __floats2bfloat162_rn(lo2f(acc[a0 + k]), hi2f(acc[a0 + k]));
                h[k] = *reinterpret_cast<const uint32_t*>(&two);
              }
              w = make_uint4(h[0], h[1], h[2], h[3]);
            } else {
              w = make_uint4(__float_as_uint(lo2f(acc[a0])), __float_as_uint(hi2f(acc[a0])), __float_as_uint(lo2f(acc[a0 + 1])),
                             __float_as_uint(hi2f(acc[a0 + 1])));
            }
            *reinterpret_cast<uint4*>(staged + lane * kPitch + 16 * j) = w;
          }
          __syncwarp();
          const int n = n0 * 256 + eg * 128 + piece * C;
          if constexpr (VEC) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int r = 4 * j + (lane >> 3), m = n + (lane & 7) * E;
              const uint4 w = *reinterpret_cast<const uint4*>(staged + r * kPitch + 16 * (lane & 7));
              if (!(valid_rows >> r & 1)) continue;
              OUT* dst = static_cast<OUT*>(p.out) + (long long)(wrow0 + r) * p.os + m;
              if (m + E <= p.N) {
                *reinterpret_cast<uint4*>(dst) = w;
              } else {
                const OUT* e = reinterpret_cast<const OUT*>(&w);
#pragma unroll
                for (int k = 0; k < E; ++k)
                  if (m + k < p.N) dst[k] = e[k];
              }
            }
          } else {
            store_rows(static_cast<OUT*>(p.out) + (long long)wrow0 * p.os + n, p.os, staged, valid_rows, p.N - n);
          }
          __syncwarp();
        }
      }
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (warp == 1 && rank == 1) tc::mbar_wait_warp(done, 0, p.status);  // the last commit's arrival, behind all others', before the barriers go
  tc::cluster_sync_all();  // no copy, commit, arrival or product of the pair is outstanding past this point
  if (warp == 1) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <bool GATED, typename OUT, bool VEC>
cudaError_t launch(const fp8::Operands& o, const ProductArgs& p, int row_tiles, int tiles, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(fp8_pair_kernel<GATED, OUT, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  fp8::Maps m;
  if (!fp8::make_maps(m, o, p, 128, GATED ? 64 : 128)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * std::min(tiles, std::max(1, device_sms() / 2)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fp8_pair_kernel<GATED, OUT, VEC>, m.x, m.w0, m.w1, p, row_tiles, tiles);
}

}  // namespace

namespace fp8 {

// 0.43 us a k block of a tile, 3 us to start and end. 512 rows: 6,144 x 4,096 16.6 us, with the few-row kernel 19.4; 4,096 x 12,288 37.7 us, 28.0 with
// it, since 32 tiles leave most SMs idle. Gated 12,288 x 4,096: 256 rows 32.9 us, 44.5 with it; 128 rows, which fill half of a tile, 34.5 and
// 25.7: up to 128 rows this kernel is not asked.
double pairs_us(const ProductArgs& p, bool gated) {
  const int pairs = std::max(1, device_sms() / 2);
  const long long tiles = (long long)((p.rows + 255) / 256) * (gated ? blocks_of(p.N) : (p.N + 255) / 256);
  return 3.0 + 0.43 * (double)((tiles + pairs - 1) / pairs) * p.kblocks;
}

cudaError_t launch_pairs(const Operands& o, const ProductArgs& p, bool gated, bool f32, cudaStream_t s) {
  const int row_tiles = (p.rows + 255) / 256, tiles = row_tiles * (gated ? blocks_of(p.N) : (p.N + 255) / 256);
  if (gated) return launch<true, float, true>(o, p, row_tiles, tiles, s);
  if (!p.vec) return f32 ? launch<false, float, false>(o, p, row_tiles, tiles, s) : launch<false, bf16, false>(o, p, row_tiles, tiles, s);
  return f32 ? launch<false, float, true>(o, p, row_tiles, tiles, s) : launch<false, bf16, true>(o, p, row_tiles, tiles, s);
}

}  // namespace fp8
}  // namespace dlite
