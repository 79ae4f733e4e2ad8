// Products of 8-bit rows and 8-bit weights with a scale per block, and the gated form whose activation leaves in 8 bits again.
//
//   linear: out[r, n] = sum_b xs[r, b] ws[n / 128, b] sum_{k in block b} x[r, k] w[n, k]
//   gated:  g, u the same sums over two weights, a = silu(g) u, stored as codes with a scale per (row, 128 columns)
//
// This kernel serves few rows. A CTA computes 128 rows x 128 weight rows over a run of k blocks. Per k block four
// tcgen05.mma kind::f8f6f4 (K = 32) write an accumulator of their own in tensor memory, two in turn; the epilogue warps (lane = row) multiply it by
// the block's scales and add it to sums in registers, in float32, while the next block's products run. The k blocks of a tile are
// dealt to `splits` CTAs of one cluster, whose sums meet in shared memory: every CTA reads all parts of the rows
// that are its own, in order, so results are the same run to run.
// Gated: a tile has 64 gate rows and the 64 up rows of the same columns; two CTAs of a cluster make up the 128 columns
// that share a scale.
// Bound: the weights' bytes, and 4 us to begin and end (the way of the first bytes, the join). A graph's call, weights from HBM: 1 row of 4,096 x
// 4,096 6.4 us (floor 2.5), of 4,096 x 12,288 10.9 (7.4), 8 rows of 151,936 x 4,096 91 to 94 (91.8: 98% of the copy rate), gated 12,288 x
// 4,096 20.4 (14.9). With full row tiles the way round of an accumulator counts: 256 rows of 6,144 x 4,096 13.6 us, 0.95 PFLOP/s.
#include <algorithm>

#include "fp8.cuh"
#include "tc_device.cuh"

namespace dlite {
namespace {

using fp8::kBlock;
using fp8::ProductArgs;

constexpr int kThreads = 320;              // copy warp, MMA warp, eight epilogue warps
constexpr uint32_t kWTile = 128 * 128;     // a k block of the weights' 128 rows
constexpr uint32_t kCols = 256;            // tensor memory: two accumulators of 128 columns
constexpr int kPitch = 132;                // floats of a staged row (16-byte stores of a warp's lanes fall on different banks)
// k blocks of the weights asked into L2 before the kernel before has ended: a feed-forward block of one row, three kernels, took 37.1 us
// with none, 34.8 with four, 35.6 with eight, 36.1 with 16
constexpr int kAhead = 4;
constexpr size_t kSmem = 112 * 1024;       // two CTAs an SM

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

struct SmallPlan {
  int box;     // rows of an activation tile's copy
  int splits;  // of the k blocks
  int stages;
  uint32_t a_bytes;
};

template <bool GATED, typename OUT>
__global__ void __launch_bounds__(kThreads, 2)
    fp8_small_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw0,
                     const __grid_constant__ CUtensorMap mw1, const ProductArgs p, const SmallPlan pl) {
  // Shared memory: [barriers | pad to 1 KB] [stage 0] ..; stage = [activation tile][weight tile]. The sums of the rows are staged over the stages.
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = (uint64_t*)base;
  const uint32_t full0 = tc::su32(bars), empty0 = tc::su32(bars + pl.stages), accf0 = tc::su32(bars + 2 * pl.stages);
  const uint32_t acce0 = accf0 + 16, done = accf0 + 32;
  uint32_t* tmem_holder = (uint32_t*)(bars + 2 * pl.stages + 5);
  uint8_t* smem = base + 1024;
  const uint32_t stage_bytes = pl.a_bytes + kWTile;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int halves = GATED ? 2 : 1, cl = halves * pl.splits;
  const int rank = blockIdx.x % cl, half = GATED ? rank & 1 : 0, z = GATED ? rank >> 1 : rank;
  const int tile = blockIdx.x / cl;                              // 128 columns of the result
  const int row0 = blockIdx.y * 128, rows = min(128, p.rows - row0);
  const int kb0 = (int)((long long)z * p.kblocks / pl.splits), kn = (int)((long long)(z + 1) * p.kblocks / pl.splits) - kb0;
  const int quads = (rows + 31) / 32;                            // quarters of the accumulator's lanes that hold rows

  if (threadIdx.x == 0) {
    for (int s = 0; s < pl.stages; ++s) {
      tc::mbar_init(full0 + 8 * s, 1);
      tc::mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(accf0 + 8 * b, 1);
      tc::mbar_init(acce0 + 8 * b, 2 * quads);
    }
    tc::mbar_init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::su32(tmem_holder)), "r"(kCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    pdl_trigger();  // behind the allocation: a kernel after this one cannot take columns that it still waits for
  }
  if (warp == 0 && fp8::elect_one())
    for (int j = 0; j < min(kn, kAhead); ++j) {
      const int k = (kb0 + j) * kBlock;
      fp8::prefetch_2d(&mw0, k, tile * 128 + half * 64);
      if (GATED) fp8::prefetch_2d(&mw1, k, tile * 128 + half * 64);
    }
  pdl_wait();
  tc::fence_before();
  // a tile without a valid row (padding of a ragged batch) is left out by the whole cluster
  const bool live = __syncthreads_or((int)threadIdx.x < rows && fp8::valid_row(p.n_rows, p.T, row0 + threadIdx.x));
  tc::fence_after();
  const uint32_t tmem = *tmem_holder;
  float* staged = (float*)smem;

  if (live && warp == 0) {  // ---------------- copies
    if (fp8::elect_one()) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int j = 0; j < kn && ok; ++j) {
        if (j >= pl.stages) ok = tc::mbar_wait_hint(empty0 + 8 * s, ph ^ 1u, p.status);
        if (!ok) break;
        const uint32_t st = tc::su32(smem + (size_t)s * stage_bytes), bar = full0 + 8 * s;
        const int k = (kb0 + j) * kBlock;
        tc::mbar_expect_tx(bar, (uint32_t)pl.box * 128 + kWTile);
        if (GATED) {
          tc::tma_load_2d(st + pl.a_bytes, &mw0, bar, k, tile * 128 + half * 64);
          tc::tma_load_2d(st + pl.a_bytes + kWTile / 2, &mw1, bar, k, tile * 128 + half * 64);
        } else {
          tc::tma_load_2d(st + pl.a_bytes, &mw0, bar, k, tile * 128);
        }
        tc::tma_load_2d(st, &mx, bar, k, row0);
        if (++s == pl.stages) {
          s = 0;
          ph ^= 1u;
        }
      }
      // no copy is in flight past this role, whoever gave up
      const int last = kn < pl.stages ? kn : pl.stages;
      if (!ok)
        for (int i = 0; i < last; ++i) {
          if (s == 0) {
            s = pl.stages;
            ph ^= 1u;
          }
          --s;
          tc::mbar_wait_hint(full0 + 8 * s, ph, p.status);
        }
    }
    __syncwarp();
  } else if (live && warp == 1) {  // ---------------- products
    if (fp8::elect_one()) {
      constexpr uint32_t idesc = fp8::idesc_e4m3(128, 128);
      int s = 0;
      uint32_t ph = 0;
      for (int j = 0; j < kn; ++j) {
        const int b = j & 1;
        if (j >= 2 && !tc::mbar_wait_hint(acce0 + 8 * b, (uint32_t)((j >> 1) - 1) & 1u, p.status)) break;
        if (!tc::mbar_wait_hint(full0 + 8 * s, ph, p.status)) break;
        tc::fence_after();
        const uint64_t a0 = tc::sw128_desc(tc::su32(smem + (size_t)s * stage_bytes)), b0 = a0 + (pl.a_bytes >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) fp8::umma_e4m3(tmem + 128 * b, a0 + 2 * kk, b0 + 2 * kk, idesc, kk > 0);
        tc::umma_commit(accf0 + 8 * b);
        tc::umma_commit(empty0 + 8 * s);
        if (++s == pl.stages) {
          s = 0;
          ph ^= 1u;
        }
      }
      // every product issued has finished before the stages and the tensor memory go
      tc::umma_commit(done);
      tc::mbar_wait_hint(done, 0, p.status);
    }
    __syncwarp();
  } else if (live && (warp & 3) < quads) {  // ---------------- sums: lane = row, 64 columns a thread
    const int q = warp & 3, eg = (warp - 2) >> 2, r = q * 32 + lane;
    const float* xs = p.xs + (long long)kb0 * p.rows + row0 + min(r, rows - 1);
    const float* ws = (GATED && eg ? p.ws[1] : p.ws[0]) + (long long)tile * p.kblocks + kb0;
    uint64_t acc[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[i] = 0;
    float x = xs[0], w = ws[0];
    bool ok = true;
    for (int j = 0; j < kn; ++j) {
      const int b = j & 1;
      const float sc = x * w;
      const uint64_t sc2 = pack2f(sc, sc);
      if (j + 1 < kn) {
        xs += p.rows;
        x = *xs;
        w = ws[j + 1];
      }
      ok = fp8::wait_all(accf0 + 8 * b, (uint32_t)(j >> 1) & 1u, p.status);
      if (!ok) break;
      tc::fence_after();
      const uint32_t t0 = tmem + ((uint32_t)(q * 32) << 16) + 128 * b + 64 * eg;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t v[16];
        tc::tmem_ld16_nowait(t0 + 16 * c, v);
        tc::tmem_wait_ld();
        if (c == 3) {  // all read: the accumulator is the products' again
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(acce0 + 8 * b);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          acc[8 * c + i] = fma2(pack2f(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), sc2, acc[8 * c + i]);
      }
    }
    // the last accumulator is there, so every product has read its stage: their memory takes the sums
    if (ok && r < rows) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        *reinterpret_cast<float4*>(staged + r * kPitch + 64 * eg + 4 * i) =
            make_float4(lo2f(acc[2 * i]), hi2f(acc[2 * i]), lo2f(acc[2 * i + 1]), hi2f(acc[2 * i + 1]));
    }
  }
  tc::fence_before();
  __syncthreads();
  if (cl > 1) tc::cluster_sync_all();
  if (warp == 1) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
  }
  if (live) {  // ---------------- the rows of the tile, dealt to the cluster's warps
    const uint32_t mine = tc::su32(staged);
    auto part = [&](int rk, int r, int c) { return ld_cluster4(tc::map_to_rank(mine, rk) + (uint32_t)(r * kPitch + c) * 4); };
    for (int r = rank + cl * warp; r < rows; r += cl * (kThreads / 32)) {
      const int row = row0 + r;
      if (!fp8::valid_row(p.n_rows, p.T, row)) continue;
      if constexpr (GATED) {
        const int hf = lane >> 4, c = (lane & 15) * 4, n = tile * 128 + hf * 64 + c;
        float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
        for (int i = 0; i < pl.splits; ++i) {
          const float4 a = part(2 * i + hf, r, c), b = part(2 * i + hf, r, 64 + c);
          g.x += a.x, g.y += a.y, g.z += a.z, g.w += a.w;
          u.x += b.x, u.y += b.y, u.z += b.z, u.w += b.w;
        }
        const uint64_t a0 = fp8::gated2(pack2f(g.x, g.y), pack2f(u.x, u.y)), a1 = fp8::gated2(pack2f(g.z, g.w), pack2f(u.z, u.w));
        float v[4] = {lo2f(a0), hi2f(a0), lo2f(a1), hi2f(a1)};
        bool bad = false;
        const float amax = warp_max(fp8::finite_max(v, bad));   // columns past N are 0
        const int e = fp8::block_exponent(amax);
        const float inv = fp8::exp2i(-e);
        const uint32_t w = fp8::codes4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
        uint8_t* dst = p.codes + (long long)row * p.cs + n;
        if (n + 4 <= p.N)
          *reinterpret_cast<uint32_t*>(dst) = w;
        else
          for (int i = 0; i < p.N - n; ++i) dst[i] = (uint8_t)(w >> (8 * i));
        if (lane == 0) p.scale[(long long)tile * p.rows + row] = fp8::exp2i(e);
        if (bad) flag_status(p.status, kDevNonfinite);
      } else {
        const int n = tile * 128 + lane * 4;
        float4 o = part(0, r, lane * 4);
        for (int i = 1; i < pl.splits; ++i) {
          const float4 a = part(i, r, lane * 4);
          o.x += a.x, o.y += a.y, o.z += a.z, o.w += a.w;
        }
        OUT* dst = static_cast<OUT*>(p.out) + (long long)row * p.os + n;
        const float v[4] = {o.x, o.y, o.z, o.w};
        OUT e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (sizeof(OUT) == 2)
            e[i] = __float2bfloat16_rn(v[i]);
          else
            e[i] = v[i];
        }
        if (p.vec && n + 4 <= p.N) {
          if constexpr (sizeof(OUT) == 2)
            *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(e);
          else
            *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(e);
        } else {
          for (int i = 0; i < 4; ++i)
            if (n + i < p.N) dst[i] = e[i];
        }
      }
    }
  }
  if (cl > 1) tc::cluster_sync_all();  // no CTA's sums go while another reads them
}

// ---------------------------------------------------------------- host side

// Splits of the k blocks: the least time of one CTA's run, where two CTAs on an SM take 8/5 of one's time a block (1 row, 4,096 x
// 12,288: 4 splits, 128 CTAs, 12.1 us, 8 splits, 256 CTAs, 10.9; 32 rows, 6,144 x 4,096: 3 splits, 144 CTAs, 8.7, 4 splits, 192 CTAs, 9.0). At
// least four blocks a CTA (340 rows, 1,024 x 2,176: 8.0 us with four, 9.7 with two), and clusters of four and more leave an eighth of the
// places free, since not every GPC has a multiple of them (gated 9,728 x 2,560, 8 rows: 152 CTAs in twos 11.7 us, 304 in fours 16.5).
// us: an estimate of the call's time, to be compared with the many-row kernel's.
SmallPlan small_plan(const ProductArgs& p, bool gated, double& us) {
  SmallPlan pl;
  pl.box = p.rows >= 128 ? 128 : (p.rows + 7) / 8 * 8;
  pl.a_bytes = (uint32_t)(pl.box * 128);
  pl.stages = std::min<int>(16, (int)((kSmem - 2048) / (pl.a_bytes + kWTile)));
  const int halves = gated ? 2 : 1, sms = device_sms();
  const long long tiles = (long long)fp8::blocks_of(p.N) * halves * ((p.rows + 127) / 128);
  pl.splits = 1;
  double best = 0;
  for (int s : {1, 2, 3, 4, 6, 8}) {
    const long long ctas = tiles * s, places = halves * s >= 4 ? 2LL * sms * 7 / 8 : 2LL * sms;
    const int run = (p.kblocks + s - 1) / s;
    if (s > 1 && (halves * s > 8 || run < 4 || ctas > places)) break;
    const double t = (double)((ctas + 2 * sms - 1) / (2 * sms)) * run * (ctas <= sms ? 5 : 8);
    if (s == 1 || t < best) {
      best = t;
      pl.splits = s;
    }
  }
  // full row tiles: 0.5 us a block alone on an SM, 0.6 two at a time for both; 4.5 us to start, join and end
  us = 4.5 + best * (tiles * pl.splits <= sms ? 0.5 / 5 : 0.6 / 8);
  return pl;
}

template <bool GATED, typename OUT>
cudaError_t launch_small(const fp8::Operands& o, const ProductArgs& p, const SmallPlan& pl, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(fp8_small_kernel<GATED, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  fp8::Maps m;
  if (!fp8::make_maps(m, o, p, pl.box, GATED ? 64 : 128)) return cudaErrorInvalidValue;
  const int cl = (GATED ? 2 : 1) * pl.splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(fp8::blocks_of(p.N) * cl, (p.rows + 127) / 128);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fp8_small_kernel<GATED, OUT>, m.x, m.w0, m.w1, p, pl);
}

template <bool GATED, typename OUT>
int product(const ProductArgs& p, const fp8::Operands& o, cudaStream_t s) {
  double us;
  const SmallPlan pl = small_plan(p, GATED, us);
  if (p.rows > 128 && fp8::pairs_us(p, GATED) < us) return launch_status(fp8::launch_pairs(o, p, GATED, sizeof(OUT) == 4, s));
  return launch_status(launch_small<GATED, OUT>(o, p, pl, s));
}

}  // namespace

namespace fp8 {

bool make_maps(Maps& m, const Operands& o, const ProductArgs& p, int x_box, int w_box) {
  typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? (Encode)f : (Encode) nullptr;
  }();
  if (!fn) return false;
  auto map = [&](CUtensorMap* to, const void* base, int rows, long long stride, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)p.K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {(cuuint32_t)kBlock, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return fn(to, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (!map(&m.x, o.x, p.rows, o.xs, x_box) || !map(&m.w0, o.w[0], p.N, o.ws[0], w_box)) return false;
  if (o.w[1]) return map(&m.w1, o.w[1], p.N, o.ws[1], w_box);
  m.w1 = m.w0;
  return true;
}

}  // namespace fp8
}  // namespace dlite

namespace {

// What both products check of their operands.
int check_product(int B, int T, int K, int N, const void* codes, int64_t codes_stride, const float* scale, const int32_t* n_rows, const int* status) {
  if (!codes || !scale || B < 1 || T < 1 || K < 1 || N < 1) return DLITE_ERR_INVALID_ARG;
  if (((uintptr_t)codes & 15) || codes_stride < K || codes_stride % 16 || !dlite::aligned4(scale, n_rows, status)) return DLITE_ERR_INVALID_ARG;
  if ((long long)B * T > DLITE_FP8_MAX_ROWS || K > DLITE_FP8_MAX_K || N > DLITE_FP8_MAX_N || codes_stride >= (1LL << 40)) return DLITE_ERR_UNSUPPORTED_SHAPE;
  return DLITE_OK;
}
// The scales of `rows` rows (of a weight: of blocks of rows) of K columns, which are dense
dlite::Rows scales(const float* at, int rows, int K) { return {at, 1, 0, 4LL * rows * dlite::fp8::blocks_of(K)}; }
int check_weight(const void* w, int64_t stride, const float* scale, int K) {
  if (!w || !scale || ((uintptr_t)w & 15) || stride < K || stride % 16 || ((uintptr_t)scale & 3)) return DLITE_ERR_INVALID_ARG;
  return stride >= (1LL << 40) ? DLITE_ERR_UNSUPPORTED_SHAPE : DLITE_OK;
}

}  // namespace

extern "C" int dlite_fp8_linear(const dlite_fp8_linear_args* g, dlite_stream_t stream) {
  using namespace dlite;
  if (!g) return DLITE_ERR_INVALID_ARG;
  if (const int rc = check_product(g->B, g->T, g->K, g->N, g->codes, g->codes_stride, g->scale, g->n_rows, g->status)) return rc;
  if (const int rc = check_weight(g->w, g->w_stride, g->w_scale, g->K)) return rc;
  if (g->dtype != DLITE_F32 && g->dtype != DLITE_BF16) return DLITE_ERR_INVALID_ARG;
  const int es = g->dtype == DLITE_F32 ? 4 : 2;
  if (!g->out || (uintptr_t)g->out % es || g->out_stride < g->N) return DLITE_ERR_INVALID_ARG;
  ProductArgs p = {};
  p.rows = g->B * g->T;
  p.T = g->T;
  p.K = g->K;
  p.kblocks = fp8::blocks_of(g->K);
  p.N = g->N;
  p.n_rows = g->n_rows;
  p.xs = g->scale;
  p.ws[0] = p.ws[1] = g->w_scale;
  p.out = g->out;
  p.os = g->out_stride;
  p.vec = !((uintptr_t)g->out & 15) && g->out_stride % (16 / es) == 0;
  p.status = g->status;
  const cudaStream_t s = (cudaStream_t)stream;
  if (!apart_of(Rows{p.out, p.rows, p.os * es, (long long)p.N * es}, Rows{g->codes, p.rows, g->codes_stride, p.K}, scales(p.xs, p.rows, p.K),
                Rows{g->w, p.N, g->w_stride, p.K}, scales(p.ws[0], fp8::blocks_of(p.N), p.K)))
    return DLITE_ERR_INVALID_ARG;
  const fp8::Operands o = {g->codes, g->codes_stride, {g->w, nullptr}, {g->w_stride, 0}};
  return g->dtype == DLITE_F32 ? product<false, float>(p, o, s) : product<false, bf16>(p, o, s);
}

extern "C" int dlite_fp8_gated(const dlite_fp8_gated_args* g, dlite_stream_t stream) {
  using namespace dlite;
  if (!g) return DLITE_ERR_INVALID_ARG;
  if (const int rc = check_product(g->B, g->T, g->K, g->F, g->codes, g->codes_stride, g->scale, g->n_rows, g->status)) return rc;
  if (const int rc = check_weight(g->gate, g->gate_stride, g->gate_scale, g->K)) return rc;
  if (const int rc = check_weight(g->up, g->up_stride, g->up_scale, g->K)) return rc;
  if (!g->out_codes || ((uintptr_t)g->out_codes & 15) || g->out_stride < g->F || g->out_stride % 16 || !g->out_scale || ((uintptr_t)g->out_scale & 3))
    return DLITE_ERR_INVALID_ARG;
  ProductArgs p = {};
  p.rows = g->B * g->T;
  p.T = g->T;
  p.K = g->K;
  p.kblocks = fp8::blocks_of(g->K);
  p.N = g->F;
  p.n_rows = g->n_rows;
  p.xs = g->scale;
  p.ws[0] = g->gate_scale;
  p.ws[1] = g->up_scale;
  p.codes = g->out_codes;
  p.cs = g->out_stride;
  p.scale = g->out_scale;
  p.status = g->status;
  const Rows codes = {p.codes, p.rows, p.cs, p.N}, scale = scales(p.scale, p.rows, p.N);
  for (const Rows& out : {codes, scale})
    if (!apart_of(out, Rows{g->codes, p.rows, g->codes_stride, p.K}, scales(p.xs, p.rows, p.K), Rows{g->gate, p.N, g->gate_stride, p.K},
                  scales(p.ws[0], fp8::blocks_of(p.N), p.K), Rows{g->up, p.N, g->up_stride, p.K}, scales(p.ws[1], fp8::blocks_of(p.N), p.K)))
      return DLITE_ERR_INVALID_ARG;
  if (!apart(codes, scale)) return DLITE_ERR_INVALID_ARG;
  const fp8::Operands o = {g->codes, g->codes_stride, {g->gate, g->up}, {g->gate_stride, g->up_stride}};
  return product<true, float>(p, o, (cudaStream_t)stream);
}
