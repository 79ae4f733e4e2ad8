// Attention over the paged 4-bit cache on the tcgen05 tensor cores: bf16 queries, heads of 128.
//
// A unit is a tile of 128 keys (two pages) of one KV head. The keys are the rows of the first product and the columns of a head
// the rows of the second, so both cached operands are A operands, and those can come from tensor memory:
//   S^T [128 keys x N rows] = K [128 x 128] Q^T,   O^T [128 columns x N rows] += V^T [128 x 128 keys] P^T.
// A thread of the dequantising warps owns one lane of tensor memory: one key (its 64 bytes of codes, 8 scales) or one
// column (its 64 bytes of codes along the tokens, the scales of 128 tokens). It turns its codes into f16 (e2m1 x e4m3 is exact)
// and writes them with tcgen05.st, so the cache never passes through shared memory a second time. N = 16 or 32
// query rows; Q^T and P^T are the B operands in shared memory.
// Warps: 0-3 keys, 4-7 values, 8-15 softmax and output (thread = key, then column), 16 value scales to f16, 17 and 18 the issue
// of the first and the second product, 19 copies: five warps a scheduler.
// The softmax warps are two groups that take the tiles in turn, each with its own scores, weights, maxima, sums and O, joined at
// a piece's end: one group's latencies pass under the other's tile (one group alone took 3,300 clocks a tile). A group keeps one
// reference m per row, a raw score, moved only when a weight passes it by more than 2^8 (a vote of its four warps per tile); only then
// are exact maxima formed and O, the sums rescaled. Weights are 2^((s - m) factor + 6) <= 2^14, rounded to f16: weights down
// to 2^-31 of the reference count, and the largest score is never below it. The sums are of the weights before that rounding, in
// fp32, a thread's own in tensor memory: 32 more registers spilled (67 us, then, for 52), and a product of the rounded weights
// with ones was 3 us faster but its lse off by more than 10^-6. Queries are scaled by a power of two per
// row into f16's range: exact for bf16 elements down to 2^-32 of the row's largest, and off by 2^-39 of that below. (One power of two
// per tile saves the loads of the factors, 4% of the ragged batch, but a row beside much larger ones lost its bits; both, by a branch per tile: no faster.)
// The issuing warps stay converged and elect a lane: 17 clocks an MMA, 46 from a branch on the lane (the operands then
// go from vector to uniform registers one by one).
// Bound: the chain of a softmax group's tile (scores out of tensor memory, vote, exponentials, weights to shared memory, sums), of which two groups
// in turn hide half. A tile of 128 keys takes 1,100 clocks at N = 16 and 1,460 at N = 32 (from the slope between 118,000 and 236,000 keys);
// its 18 KB take 795 at the copy rate of HBM, its warp instructions at most 820 and 1,040 of a scheduler's slots (75% and 70%; 256 of them
// convert codes), the tensor pipe is active for 13%. Twice the dequantising warps (28 in all, registers shared out again with setmaxnreg)
// changed nothing, nor did 9 or 10 stages for 8. Around the
// tiles: 6 us up to the first weights (lengths, list of pieces, first records, first maxima), 1.5 us at the end, 4 us the
// join with its launch; a change of pieces costs a CTA 8 tiles.
// Measured (32 query heads, 8 KV heads, with the join): one request of 118,000 keys 40 us for one token, 54 us for eight; eight requests
// of 8,192 keys, one token each, 21 us; 32 requests of up to 40,960 keys, up to eight tokens each, 224 us (49% of the copy rate).
// mma.sync does both products of a 32-row tile in 8 clocks a key an SM (measured 2.0 per m16n8k16), above the 6.8 that the bytes take
// at the copy rate of HBM, and needs its operands and outputs in registers: the mma.sync kernel ran at 19.
#include <math.h>

#include <type_traits>

#include "kv_attention.cuh"
#include "tc_gemm.h"

namespace dlite {
namespace kv {
namespace {

constexpr int DH = 128, REC = rec_bytes(DH), TILE = 2 * REC;
constexpr int kStages = 8;
constexpr int kThreads = 20 * 32;
// A tile's flags and the barrier of its value scales, which the softmax looks at last: the copies and scales of tile i + 16 take
// the stage of i + 8, whose values take the buffer of i + 6, whose second product comes after the softmax of i + 6 and so of i.
constexpr int kRing = 2 * kStages;
// A stage holds both pages' records as they are, one copy each, as rows of 128 bytes under a 128-byte swizzle.
constexpr int kRow = 128, kRecRows = REC / kRow;
static_assert(REC % 1024 == 0 && kRecRows <= 256, "rows of a copy");
// 16-byte chunk c of a record
__device__ __forceinline__ int chunk(int c) { return c / 8 * kRow + (((c ^ (c >> 3)) & 7) << 4); }
// tensor memory columns: K and V^T tiles twice; then S^T, O^T and the threads' sums twice each
constexpr int kTmK = 0, kTmV = 128, kTmS = 256, kTmCols = 512;
constexpr float kNoRef = -1e30f;   // reference of a row that has seen no key: raw scores are below 2^36

template <int N>
struct Smem {
  static constexpr int Q = kStages * TILE;           // [2 halves][N rows][128 B], 128-byte swizzle
  static constexpr int P = Q + N * 256;              // [2][128 keys][N rows] f16, rows of N contiguous
  static constexpr int VS = P + 2 * 128 * N * 2;     // [stage][8 blocks][128 tokens] f16: value scales
  static constexpr int ROWS = VS + kStages * 2048;         // floats: reference [2][N], alpha [2][N], l [2][N], red [2][4][N], factor [N]
  static constexpr int KEYS = ROWS + 21 * N * 4;  // int2: keys a row sees
  static constexpr int OUT = KEYS + N * 8;           // int64: where a row's output and lse go
  static constexpr int BARS = OUT + N * 16;
  static constexpr int NBARS = 2 * kStages + 17 + kRing;
  static constexpr int OK = BARS + NBARS * 8;        // [kRing]: which of a tile's pages came
  static constexpr int TM = OK + kRing * 4;
  static constexpr int LIST = (TM + 16 + 15) / 16 * 16;   // PieceTile [kBatch], then their number
  static constexpr int PREFIX = LIST + kBatch * (int)sizeof(PieceTile) + 8;
  static constexpr int BYTES = PREFIX + (kMaxList + 1) * 4 + 1024;  // alignment of the swizzled stages
  static_assert(BYTES <= 227 * 1024, "shared memory of one CTA");
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// N columns of this warp's 32 lanes; complete on return
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[N]) {
  uint32_t r[N / 16][16];
#pragma unroll
  for (int i = 0; i < N / 16; ++i) tc::tmem_ld16_nowait(addr + 16 * i, r[i]);
  tc::tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i / 16][i % 16]);
}
// 8 or 16 columns
template <int M>
__device__ __forceinline__ void tmem_ld_part(uint32_t addr, float (&v)[M]) {
  if constexpr (M == 16) {
    tmem_ld<16>(addr, v);
  } else {
    static_assert(M == 8, "rows of a group");
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
    tc::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
  }
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t addr, const float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N / 16; ++i) {
    uint32_t r[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(v[16 * i + e]);
    tmem_st16(addr + 16 * i, r);
  }
}
// D (tensor memory) (+)= A (tensor memory) B (shared memory)
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
// f16 operands, fp32 accumulator; B with its rows contiguous along N where b_mn
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// P^T as B operand, N contiguous: 8 keys of N x 2 bytes form one swizzle atom, atoms follow each other along the keys
template <int N>
__device__ __forceinline__ uint64_t p_desc(uint32_t saddr) {
  constexpr uint32_t atom = 8 * N * 2;
  constexpr uint64_t swizzle = N == 32 ? 4 : 6;  // 64 or 32 bytes
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(atom >> 4) << 16) | ((uint64_t)(atom >> 4) << 32) | ((uint64_t)1 << 46) |
         (swizzle << 61);
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(z)
      : "memory");
}
__device__ __forceinline__ void group_barrier(int g) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + g) : "memory"); }
__device__ __forceinline__ void softmax_barrier() { asm volatile("barrier.cta.sync 3, 256;" ::: "memory"); }
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Sums of N rows over a warp: the halves of the rows change sides step by step; lane i returns row i (N = 16: i / 2).
template <int N>
__device__ __forceinline__ float warp_row_sums(float (&v)[N], int lane) {
  auto step = [&](auto cnt_c, int o) {
    constexpr int cnt = decltype(cnt_c)::value;
    const bool up = lane & o;
#pragma unroll
    for (int r = 0; r < cnt; ++r) {
      const float give = up ? v[r] : v[r + cnt], keep = up ? v[r + cnt] : v[r];
      v[r] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  };
  step(std::integral_constant<int, N / 2>(), 16);
  step(std::integral_constant<int, N / 4>(), 8);
  step(std::integral_constant<int, N / 8>(), 4);
  step(std::integral_constant<int, N / 16>(), 2);
  if constexpr (N == 32) {
    step(std::integral_constant<int, 1>(), 1);
    return v[0];
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}
// A wait that did not end at once: sleep and look again, up to the limit. Then the status says so, and *gave_up ends this wait
// and every later one of the CTA: the roles run to their ends on whatever the buffers hold.
__device__ __noinline__ void wait_slow(uint32_t bar, uint32_t parity, volatile int* gave_up, int* status) {
  const uint64_t t0 = tc::gtimer();
  while (!*gave_up) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(100000u)
        : "memory");
    if (ok) return;
    if (tc::gtimer() - t0 > tc::kTimeoutNs) {
      flag_status(status, kDevTimeout);
      *gave_up = 1;
    }
  }
}
__device__ __forceinline__ void wait_phase(uint32_t bar, uint32_t parity, volatile int* gave_up, int* status) {
  if (!tc::mbar_try(bar, parity)) wait_slow(bar, parity, gave_up, status);
  __syncwarp();
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attention_tc_kernel(const __grid_constant__ CUtensorMap map, const AttnArgs a) {
  using S = Smem<N>;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024 - (tc::su32(raw) & 1023)) & 1023);
  const uint32_t sb = tc::su32(sm);
  float* rows_f = reinterpret_cast<float*>(sm + S::ROWS);
  auto row_ref = [&](int g) { return rows_f + g * N; };              // references, raw scores
  auto row_alpha = [&](int g) { return rows_f + (2 + g) * N; };
  auto row_l = [&](int g) { return rows_f + (4 + 4 * g) * N; };      // [warp][row]
  auto row_red = [&](int g) { return rows_f + (12 + 4 * g) * N; };   // [warp][row]
  float* row_sc = rows_f + 20 * N;                                   // factors of the raw scores
  int2* row_keys = reinterpret_cast<int2*>(sm + S::KEYS);
  long long* row_out = reinterpret_cast<long long*>(sm + S::OUT);  // [row] of out, [N + row] of lse
  int* stage_ok = reinterpret_cast<int*>(sm + S::OK);
  uint32_t* tm_slot = reinterpret_cast<uint32_t*>(sm + S::TM);
  int* prefix = reinterpret_cast<int*>(sm + S::PREFIX);
  PieceTile* list = reinterpret_cast<PieceTile*>(sm + S::LIST);
  int* listed = reinterpret_cast<int*>(list + kBatch);
  const uint32_t bars = sb + S::BARS;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kStages + s); };
  auto bar = [&](int kind, int buf) { return bars + 8 * (2 * kStages + 2 * kind + buf); };
  enum { kReady, kFree, vReady, vFree, sFull, sFree, pReady };   // each twice; then q_ready, voted twice, a tile's value scales
  volatile int* gave_up = reinterpret_cast<volatile int*>(sm + S::TM + 4);
  volatile int* move_ref = gave_up + 1;   // [group]: a weight of the tile passes its reference by too much
  const uint32_t q_ready = bars + 8 * (2 * kStages + 14);
  auto voted = [&](int g) { return bars + 8 * (2 * kStages + 15 + g); };
  auto c_ready = [&](int i) { return bars + 8 * (2 * kStages + 17 + i % kRing); };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(full(s), 1);
      tc::mbar_init(empty(s), 8);  // a warp of keys or values each
    }
    for (int i = 0; i < kRing; ++i) tc::mbar_init(c_ready(i), 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(kReady, i), 4);
      tc::mbar_init(bar(kFree, i), 1);
      tc::mbar_init(bar(vReady, i), 4);
      tc::mbar_init(bar(vFree, i), 1);  // the second product is done: V tile, P tile and O
      tc::mbar_init(bar(sFull, i), 1);
      tc::mbar_init(bar(sFree, i), 4);
      tc::mbar_init(bar(pReady, i), 4);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(voted(i), 4);
      move_ref[i] = 0;
    }
    *gave_up = 0;
    tc::mbar_init(q_ready, 8);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map)) : "memory");
  }
  pdl_wait();  // what is above reads nothing that the stream writes and takes nothing that the kernel before may still need
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::su32(tm_slot)), "r"(kTmCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (a.stream) build_prefix<N>(a, prefix);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = *tm_slot;
  constexpr uint32_t tmO = kTmS + 2 * N, tmL = kTmS + 4 * N;
  static_assert(tmL + 2 * N <= kTmCols, "tensor memory");

  Pieces<N> walk(a, prefix);  // thread 0's
  int it = 0;  // tiles so far, over all pieces: buffer it & 1, stage it % kStages of turn it / kStages
  // Wait until a buffer (or stage) has been filled for its `turn`-th use.
  auto wait_turn = [&](uint32_t b, int turn) { wait_phase(b, (uint32_t)turn & 1u, gave_up, a.status); };
  // ... until its use before the `turn`-th is over: nothing to wait for in the first
  auto wait_left = [&](uint32_t b, int turn) {
    if (turn) wait_turn(b, turn - 1);
  };

  int l_pieces = 0;  // pieces whose queries the first product's warp has waited for
  int2 join = make_int2(0, 0);
#pragma unroll 1
  while (true) {
    if (tid == 0) {
      int n = 0;
      while (n < kBatch && walk.next(list[n].p)) ++n;
      *listed = n;
      if (n && a.stream) join = walk.join_of(true, list[n - 1].p);
    }
    __syncthreads();
    const int batch = *listed;
    if (tid < batch) {
      PieceTile& x = list[tid];
      x.b = x.p.j / a.row_tiles;
      x.rt = x.p.j - x.b * a.row_tiles;
      x.t = tile_of<N>(a, x.b, x.rt);
    }
    __syncthreads();
    if (!batch) break;
    if (warp < 4) {  // ---------------------------------------------------------------- keys
      const int page = warp >> 1, row = 32 * (warp & 1) + lane;  // key 32 warp + lane of the tile
#pragma unroll 1
      for (int k = 0; k < batch; ++k) {
        const Piece pc = list[k].p;
#pragma unroll 1
        for (int u = pc.u0; u < pc.u1; ++u, ++it) {
          const int buf = it & 1, st = it % kStages;
          wait_turn(full(st), it / kStages);
          wait_left(bar(kFree, buf), it >> 1);
          tc::fence_after();
          const uint8_t* stage = sm + st * TILE;
          const uint8_t* rec = stage + page * REC;
          const uint2 sc = *reinterpret_cast<const uint2*>(rec + chunk(ks_off(DH) / 16 + (row >> 1)) + 8 * (row & 1));
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t r[32];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint4 w = *reinterpret_cast<const uint4*>(rec + chunk(4 * row + 2 * half + q));
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
              const uint32_t s2 = fp8x2_to_f16x2((uint16_t)((half ? sc.y : sc.x) >> (16 * q)));
              const uint32_t s0 = __byte_perm(s2, s2, 0x1010), s1 = __byte_perm(s2, s2, 0x3232);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t s = i < 2 ? s0 : s1;
                r[16 * q + 4 * i] = mul_f16x2(fp4x2_of<0>(ww[i]), s);
                r[16 * q + 4 * i + 1] = mul_f16x2(fp4x2_of<1>(ww[i]), s);
                r[16 * q + 4 * i + 2] = mul_f16x2(fp4x2_of<2>(ww[i]), s);
                r[16 * q + 4 * i + 3] = mul_f16x2(fp4x2_of<3>(ww[i]), s);
              }
            }
            tmem_st32(tm + ((uint32_t)(32 * warp) << 16) + kTmK + 64 * buf + 32 * half, r);
          }
          if (lane == 0) tc::mbar_arrive(empty(st));
          __syncwarp();
          tmem_wait_st();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(kReady, buf));
        }
      }
    } else if (warp < 8) {  // ---------------------------------------------------------------- values
      const int d = 32 * (warp - 4) + lane;
#pragma unroll 1
      for (int k = 0; k < batch; ++k) {
        const Piece pc = list[k].p;
#pragma unroll 1
        for (int u = pc.u0; u < pc.u1; ++u, ++it) {
          const int buf = it & 1, st = it % kStages;
          wait_turn(c_ready(it), it / kRing);  // and the stage with them
          wait_left(bar(vFree, buf), it >> 1);
          tc::fence_after();
#pragma unroll
          for (int page = 0; page < 2; ++page) {
            const uint8_t* rec = sm + st * TILE + page * REC;
            const uint8_t* sp = sm + S::VS + st * 2048 + (d >> 4) * 256 + page * 128;
            uint32_t r[32];
#pragma unroll
            for (int q = 0; q < 2; ++q) {  // 32 tokens
              const uint4 w = *reinterpret_cast<const uint4*>(rec + chunk(v_off(DH) / 16 + 2 * d + q));
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint4 s = *reinterpret_cast<const uint4*>(sp + 64 * q + 16 * i);
                r[16 * q + 4 * i] = mul_f16x2(fp4x2_of<0>(ww[i]), s.x);
                r[16 * q + 4 * i + 1] = mul_f16x2(fp4x2_of<1>(ww[i]), s.y);
                r[16 * q + 4 * i + 2] = mul_f16x2(fp4x2_of<2>(ww[i]), s.z);
                r[16 * q + 4 * i + 3] = mul_f16x2(fp4x2_of<3>(ww[i]), s.w);
              }
            }
            tmem_st32(tm + ((uint32_t)(32 * (warp - 4)) << 16) + kTmV + 64 * buf + 32 * page, r);
          }
          if (lane == 0) tc::mbar_arrive(empty(st));
          __syncwarp();
          tmem_wait_st();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(vReady, buf));
        }
      }
    } else if (warp < 16) {  // ---------------------------------------------------------------- softmax and output
      const int g = (warp - 8) >> 2, w = warp & 3;
      const uint32_t lanes = (uint32_t)(32 * w) << 16;
      uint2 raw_q[N / 8];
      auto load_q = [&](int k) {  // rows warp - 8, + 8, ... of a piece: every load before the first use
        const Tile& t = list[k].t;
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
          const int r = t.r0 + min(warp - 8 + 8 * i, t.r1 - t.r0 - 1), tk = r / a.group, hq = list[k].p.h * a.group + r - tk * a.group;
          const bf16* q = static_cast<const bf16*>(a.q) + ((long long)list[k].b * a.T + tk) * a.qs + (long long)hq * DH + 4 * lane;
          if (a.vec) {
            raw_q[i] = *reinterpret_cast<const uint2*>(q);
          } else {
            const unsigned short* q16 = reinterpret_cast<const unsigned short*>(q);
            raw_q[i] = make_uint2(q16[0] | (uint32_t)q16[1] << 16, q16[2] | (uint32_t)q16[3] << 16);
          }
        }
      };
      load_q(0);
#pragma unroll 1
      for (int k = 0; k < batch; ++k) {
        const Piece pc = list[k].p;
        const Tile t = list[k].t;
        const int b = list[k].b, rt = list[k].rt, h = pc.h, rows = t.r1 - t.r0;
        if (warp == 8 && lane == 0 && rt == 0 && pc.u0 == 0 && (t.p0 < 0 || t.p0 + (a.n_rows ? min(a.n_rows[b], a.T) : a.T) > t.cap))
          flag_status(a.status, kDevBounds);
        // Q: all of the last piece's first products are done
        if (warp == 8 && lane < N) {
          const int r = t.r0 + lane, tk = r / a.group, hq = h * a.group + r % a.group;
          const long long row = (long long)b * a.T + tk, seen = t.p0 + tk;
          row_out[lane] = row * a.os + (long long)hq * DH;
          row_out[N + lane] = row * a.n_q + hq;
          row_keys[lane] = lane < rows ? make_int2(a.window ? (int)min(max(seen - a.window + 1, 0LL), t.cap) : 0, (int)min(max(seen + 1, 0LL), t.cap))
                                       : make_int2(0, 0);
        }
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
          const int r = warp - 8 + 8 * i;
          uint2 x = r < rows ? raw_q[i] : make_uint2(0u, 0u);
          const float v[4] = {__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                              __uint_as_float(x.y & 0xffff0000u)};
          bool q_bad = false;
          float amax = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            amax = fmaxf(amax, fabsf(v[e]));
            q_bad |= !(fabsf(v[e]) <= 3.402823466e38f);
          }
          const bool bad = __any_sync(0xffffffffu, q_bad);
          amax = warp_max_f32(amax);
          const RowScale rs = row_scale(a, bad ? 0.f : amax);
          auto f16x2 = [&](float lo, float hi) { return pack_f16(lo * rs.f0 * rs.f1, hi * rs.f0 * rs.f1); };
          x = bad ? make_uint2(0u, 0u) : make_uint2(f16x2(v[0], v[1]), f16x2(v[2], v[3]));
          // columns 4 lane ..: half lane / 16, 16-byte chunk (lane % 16) / 2 of the row, swizzled by the row
          *reinterpret_cast<uint2*>(sm + S::Q + (lane >> 4) * N * 128 + r * 128 + ((((lane >> 1) & 7) ^ (r & 7)) << 4) + 8 * (lane & 1)) = x;
          if (lane == 0) {
            row_ref(0)[r] = row_ref(1)[r] = bad ? NAN : kNoRef;
            row_sc[r] = rs.factor;
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(q_ready);
        softmax_barrier();
        const uint64_t we2 = pack2f(kTcWeightExp, kTcWeightExp);
        // tiles wholly inside every row's range need no masks
        const int full_end = (int)min(max(t.p0 + t.t_lo + 1, 0LL), t.cap);
        const int full_beg = a.window ? (int)min(max(t.p0 + t.t_hi - a.window + 1, 0LL), t.cap) : 0;
        const int first = pc.u0 + ((it ^ g) & 1);  // this group's first tile of the piece
        int last = -1;                             // its last tile so far
#pragma unroll 1
        for (int u = first; u < pc.u1; u += 2) {
          const int i = it + u - pc.u0, turn = i >> 1;
          wait_turn(bar(sFull, g), turn);
          tc::fence_after();
          const int key0 = (t.pg0 + 2 * u) * kPage, key = key0 + 32 * w + lane;
          wait_turn(c_ready(i), i / kRing);  // long over: for the flags' sake
          const int came = stage_ok[i % kRing];
          const bool masked = came != 3 || key0 < full_beg || key0 + 128 > full_end, there = (came >> (w >> 1)) & 1;
          uint64_t x[N / 2];
          auto scores = [&]() {  // -inf where the row does not see this thread's key
            float s[N];
            tmem_ld<N>(tm + lanes + kTmS + N * g, s);
            if (masked) {
#pragma unroll
              for (int r = 0; r < N; ++r) {
                const int2 see = row_keys[r];
                if (!there || key < see.x || key >= see.y) s[r] = -INFINITY;
              }
            }
#pragma unroll
            for (int r = 0; r < N / 2; ++r) x[r] = pack2f(s[2 * r], s[2 * r + 1]);
          };
          auto exponents = [&]() {
            float top = -INFINITY;
#pragma unroll
            for (int r = 0; r < N / 2; r += 2) {
              const ulonglong2 ref = *reinterpret_cast<const ulonglong2*>(row_ref(g) + 2 * r);
              const ulonglong2 sc = *reinterpret_cast<const ulonglong2*>(row_sc + 2 * r);
              x[r] = fma2(sub2(x[r], ref.x), sc.x, we2);
              x[r + 1] = fma2(sub2(x[r + 1], ref.y), sc.y, we2);
              top = fmaxf(top, fmaxf(fmaxf(lo2f(x[r]), hi2f(x[r])), fmaxf(lo2f(x[r + 1]), hi2f(x[r + 1]))));
            }
            return top;
          };
          scores();
          const bool first_tile = last < 0;  // its references are new in any case
          if (!first_tile && exponents() > kTcWeightExp + 8.f) move_ref[g] = 1;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(voted(g));
          if (!first_tile) {
#pragma unroll
            for (int r = 0; r < N / 2; ++r) x[r] = pack2f(tc::ex2_approx(lo2f(x[r])), tc::ex2_approx(hi2f(x[r])));
            wait_turn(voted(g), turn);
          }
          if (first_tile || move_ref[g]) {
            if (!first_tile) scores();
            // the exact maxima of the tile
#pragma unroll
            for (int r = 0; r < N; ++r) {
              const float mx = warp_max_f32(r & 1 ? hi2f(x[r / 2]) : lo2f(x[r / 2]));
              if (lane == r) row_red(g)[w * N + r] = mx;
            }
            group_barrier(g);
            if (w == 0 && lane < N) {
              const float* red = row_red(g);
              const float mx = fmaxf(fmaxf(red[lane], red[N + lane]), fmaxf(red[2 * N + lane], red[3 * N + lane]));
              const float ref = row_ref(g)[lane];
              row_alpha(g)[lane] = mx > ref ? tc::ex2_approx((ref - mx) * row_sc[lane]) : 1.f;
              if (mx > ref) row_ref(g)[lane] = mx;   // a NaN stays
              if (lane == 0) move_ref[g] = 0;
            }
            group_barrier(g);
            if (last >= 0) {  // O and L hold the group's tiles before this one
              wait_turn(bar(vFree, g), last >> 1);
              tc::fence_after();
#pragma unroll 1
              for (int r = 0; r < 2 * N; r += 16) {
                const uint32_t at = tm + lanes + (r < N ? tmO + N * g + r : tmL + N * g + r - N);
                float o[16];
                tmem_ld<16>(at, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= row_alpha(g)[r % N + e];
                tmem_store<16>(at, o);
              }
              tmem_wait_st();
            }
            exponents();
#pragma unroll
            for (int r = 0; r < N / 2; ++r) x[r] = pack2f(tc::ex2_approx(lo2f(x[r])), tc::ex2_approx(hi2f(x[r])));
          }
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(sFree, g));
          // P: this key's N weights side by side, once the group's last product has read the buffer
          wait_left(bar(vFree, g), turn);
          uint8_t* pp = sm + S::P + g * 128 * N * 2 + (32 * w + lane) * N * 2;
#pragma unroll
          for (int q = 0; q < N / 8; ++q) {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = pack_f16(lo2f(x[4 * q + e]), hi2f(x[4 * q + e]));
            const int sw = N == 32 ? (lane >> 1) & 3 : (lane >> 2) & 1;
            *reinterpret_cast<uint4*>(pp + ((q ^ sw) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(pReady, g));
          // this thread's keys' part of every row's sum, from the weights before their rounding
#pragma unroll
          for (int r = 0; r < N; r += 16) {
            const uint32_t at = tm + lanes + tmL + N * g + r;
            float sum[16];
            if (!first_tile) {
              tmem_ld<16>(at, sum);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) sum[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint64_t two = add2(pack2f(sum[2 * e], sum[2 * e + 1]), x[r / 2 + e]);
              sum[2 * e] = lo2f(two), sum[2 * e + 1] = hi2f(two);
            }
            tmem_store<16>(at, sum);
          }
          tmem_wait_st();
          last = i;
        }
        it += pc.u1 - pc.u0;
        if (k + 1 < batch) load_q(k + 1);
        // the groups' rows joined; thread = column 32 w + lane, group g takes rows g N / 2 ..
        if (last >= 0) {
          wait_turn(bar(vFree, g), last >> 1);
          tc::fence_after();
          float v[N];
          tmem_ld<N>(tm + lanes + tmL + N * g, v);
          const float sum = warp_row_sums<N>(v, lane);
          if (N == 32 || (lane & 1) == 0) row_l(g)[w * N + (N == 32 ? lane : lane >> 1)] = sum;
        }
        tc::fence_before();
        softmax_barrier();
        tc::fence_after();
        const int np = pc.u1 - pc.u0, r_lo = g * (N / 2);
        // whether a group had a tile: both from two tiles on, else the one whose turn the tile was
        const bool has0 = np > 1 || ((it - np) & 1) == 0, has1 = np > 1 || ((it - np) & 1) == 1;
        float L = 0.f, M = 0.f, f0 = 0.f, f1 = 0.f, inv = 0.f;  // of row `lane`
        const bool whole = pc.whole();
        if (lane < N) {
          const float r0 = row_ref(0)[lane], r1 = row_ref(1)[lane], ref = fmaxf(r0, r1), sc = row_sc[lane];
          M = ref * sc;
          f0 = has0 ? (r0 == ref ? 1.f : tc::ex2_approx((r0 - ref) * sc)) : 0.f;
          f1 = has1 ? (r1 == ref ? 1.f : tc::ex2_approx((r1 - ref) * sc)) : 0.f;
          const float *l0 = row_l(0), *l1 = row_l(1);
          L = (has0 ? f0 * (l0[lane] + l0[N + lane] + l0[2 * N + lane] + l0[3 * N + lane]) : 0.f) +
              (has1 ? f1 * (l1[lane] + l1[N + lane] + l1[2 * N + lane] + l1[3 * N + lane]) : 0.f);
          inv = whole ? (L == 0.f ? 0.f : a.v_scale / L) : 1.f;
          if (w == 0 && lane >= r_lo && lane < min(rows, r_lo + N / 2)) {
            if (!whole)
              a.part_ml[part_row(pc, N) + lane] = make_float2(M, L);
            else if (a.lse)
              a.lse[row_out[N + lane]] = lse_of(M, L, kTcWeightExp);
          }
        }
        float o0[N / 2], o1[N / 2];
#pragma unroll
        for (int r = 0; r < N / 2; ++r) o0[r] = o1[r] = 0.f;
        if (has0) tmem_ld_part<N / 2>(tm + lanes + tmO + r_lo, o0);
        if (has1) tmem_ld_part<N / 2>(tm + lanes + tmO + N + r_lo, o1);
        tc::fence_before();
        const int d = 32 * w + lane;
#pragma unroll
        for (int r = 0; r < N / 2; ++r) {
          const float e0 = __shfl_sync(0xffffffffu, f0 * inv, r_lo + r), e1 = __shfl_sync(0xffffffffu, f1 * inv, r_lo + r);
          if (r_lo + r >= rows) continue;
          const float v = fmaf(o0[r], e0, o1[r] * e1);
          if (whole)
            static_cast<bf16*>(a.out)[row_out[r_lo + r] + d] = __float2bfloat16_rn(v);
          else
            a.part_o[(part_row(pc, N) + r_lo + r) * DH + d] = v;
        }
        softmax_barrier();  // both O, row_l, row_ref are the next piece's
      }
    } else if (warp == 16) {  // ---------------------------------------------------------------- value scales
      // as f16, once for the 16 columns that share them: lane = block of 16 columns lane / 4, 32 tokens
      const int blk = lane >> 2, tok = (lane & 3) * 32;
#pragma unroll 1
      for (int k = 0; k < batch; ++k) {
        const Piece pc = list[k].p;
        const int key_end = list[k].t.key_end, pg0 = list[k].t.pg0;
#pragma unroll 1
        for (int u = pc.u0; u < pc.u1; ++u, ++it) {
          const int st = it % kStages;
          wait_turn(full(st), it / kStages);
          // keys past the end, or of a page that is not there, hold anything, a NaN scale too: their values are 0
          const int came = stage_ok[it % kRing], left = key_end - (pg0 + 2 * u) * kPage;
          const int valid = came == 3 && left >= 128 ? 32 : (came >> (tok >> 6) & 1) ? left - tok : 0;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint4 w = *reinterpret_cast<const uint4*>(sm + st * TILE + (tok >> 6) * REC + chunk(vs_off(DH) / 16 + 4 * blk + ((tok & 63) >> 4) + q));
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
            uint32_t s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              s[i] = fp8x2_to_f16x2((uint16_t)(ww[i / 2] >> (16 * (i & 1))));
              const int at = 16 * q + 2 * i;
              if (valid < 32) s[i] = at + 1 < valid ? s[i] : at < valid ? s[i] & 0xffffu : 0u;
            }
            uint4* to = reinterpret_cast<uint4*>(sm + S::VS + st * 2048 + blk * 256 + tok * 2 + 32 * q);
            to[0] = make_uint4(s[0], s[1], s[2], s[3]);
            to[1] = make_uint4(s[4], s[5], s[6], s[7]);
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(c_ready(it));
        }
      }
    } else if (warp == 19) {  // ---------------------------------------------------------------- copies
      const bool one = elect_one();
#pragma unroll 1
      for (int k = 0; k < batch; ++k) {
        const Piece pc = list[k].p;
        const Tile t = list[k].t;
        const int32_t* bt = a.bt + (size_t)list[k].b * a.max_pages + t.pg0;
        // 32 page ids at a time, the next 32 on their way: with one tile's ids loaded ahead, a load's latency was every tile's
        const int pages = min(t.np, 2 * pc.u1);
        auto page_of = [&](int i) { return i < pages ? bt[i] : -1; };
        int ids = page_of(2 * pc.u0 + lane), next_ids = page_of(2 * pc.u0 + 32 + lane);
#pragma unroll 1
        for (int u = pc.u0; u < pc.u1; ++u, ++it) {
          const int st = it % kStages;
          const int at = (2 * (u - pc.u0)) & 31;
          if (at == 0 && u > pc.u0) {
            ids = next_ids;
            next_ids = page_of(2 * u + 32 + lane);
          }
          const int id0 = __shfl_sync(0xffffffffu, ids, at), id1 = __shfl_sync(0xffffffffu, ids, at + 1);
          wait_left(empty(st), it / kStages);
          const int came = (id0 >= 0 && id0 < a.n_pages ? 1 : 0) | (id1 >= 0 && id1 < a.n_pages ? 2 : 0);
          if (one) {
            if (id0 >= a.n_pages || id1 >= a.n_pages) flag_status(a.status, kDevBounds);
            stage_ok[it % kRing] = came;
            if (came) {
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              tc::mbar_expect_tx(full(st), (came == 3 ? 2 : 1) * REC);
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                if (!(came >> p & 1)) continue;
                const long long rec = (long long)(p ? id1 : id0) * a.n_kv + pc.h;
                tma_load_3d(sb + st * TILE + p * REC, &map, full(st), (int)rec);
              }
            } else {
              tc::mbar_arrive(full(st));
            }
          }
          __syncwarp();
        }
      }
    } else if (warp == 17) {  // ---------------------------------------------------------------- first product
      const bool one = elect_one();
#pragma unroll 1
      for (int k = 0; k < batch; ++k) {
        const Piece pc = list[k].p;
        wait_turn(q_ready, l_pieces++);
#pragma unroll 1
        for (int u = pc.u0; u < pc.u1; ++u, ++it) {
          const int buf = it & 1;
          wait_turn(bar(kReady, buf), it >> 1);
          wait_left(bar(sFree, buf), it >> 1);
          tc::fence_after();
          if (one) {
            const uint64_t bd = tc::sw128_desc(sb + S::Q);
            const uint32_t ka = tm + kTmK + 64 * buf, d = tm + kTmS + N * buf;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              umma_ts(d, ka + 8 * ks, bd + (ks >> 2) * N * 8 + (ks & 3) * 2, idesc_f16(128, N, false), ks > 0);
            tc::umma_commit(bar(kFree, buf));
            tc::umma_commit(bar(sFull, buf));
          }
          __syncwarp();
        }
      }
    } else {  // ---------------------------------------------------------------- second product
      const bool one = elect_one();
#pragma unroll 1
      for (int k = 0; k < batch; ++k) {
        const Piece pc = list[k].p;
#pragma unroll 1
        for (int u = pc.u0; u < pc.u1; ++u, ++it) {
          const int buf = it & 1;
          wait_turn(bar(vReady, buf), it >> 1);
          wait_turn(bar(pReady, buf), it >> 1);
          tc::fence_after();
          if (one) {
            const uint64_t bd = p_desc<N>(sb + S::P + buf * 128 * N * 2);
            const uint32_t va = tm + kTmV + 64 * buf, o = tm + tmO + N * buf;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)  // a group's first tile of the piece starts its O
              umma_ts(o, va + 8 * ks, bd + ks * N * 2, idesc_f16(128, N, true), ks > 0 || u - pc.u0 >= 2);
            tc::umma_commit(bar(vFree, buf));
          }
          __syncwarp();
        }
      }
    }
    __syncwarp();
    __syncthreads();  // the list is the next batch's
  }
  if (tid == 0 && a.stream) a.joins[blockIdx.x] = join;
  pdl_trigger();  // late: the grid fills the SMs
  // every role is through; after a wait that ran out (status flagged) the copies and products in flight have had its time
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(kTmCols) : "memory");
}

template <int N>
cudaError_t launch(const CUtensorMap& map, const AttnArgs& a, int grid, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kv_attention_tc_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<N>::BYTES);
  return e != cudaSuccess ? e : launch_pdl(kv_attention_tc_kernel<N>, dim3(grid), dim3(kThreads), Smem<N>::BYTES, s, map, a);
}

}  // namespace

cudaError_t launch_attention_tc(const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
  CUtensorMap map;
  const long long records = (long long)a.n_pages * a.n_kv;
  if (!tc::make_record_map(&map, a.pages, kRecRows, records)) return cudaErrorInvalidValue;
  return p.rows == 16 ? launch<16>(map, a, p.grid, s) : launch<32>(map, a, p.grid, s);
}

}  // namespace kv
}  // namespace dlite
