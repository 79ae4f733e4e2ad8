// Log probabilities of given tokens, entropy and the top alternatives of rows of
// logits, in one pass over the row.
//
// With m the row's largest logit and d_v = (m - x_v) / T >= 0: S = sum e^-d, log p(v) = -d_v - log S,
// H = log S + (sum e^-d d) / S; every term is >= 0, so nothing cancels. The largest
// elements' own ones are counted apart (n) from the other terms (s), and log S = log1p(s + n - 1):
// a row that is nearly certain keeps its small entropy to full precision.
//
// A row is read by a cluster of CTAs (one when there are many rows), each a slice, each thread
// every blockDim-th 16-byte piece of the slice. The slice comes by bulk copies through a ring of shared-memory
// stages (four pieces a thread each), so that loads are in flight while a warp computes. A warp shares its running maximum m (one
// warp-wide maximum per 16 elements a lane), so that rescaling is a branch the whole warp takes, about ln(steps) times:
// with a maximum per thread some lane of a warp rescaled in most steps (512 bf16 rows of 151,936: 93.5 us). A thread
// keeps (n, s, w = sum e^-d d) and the largest of its own elements.
// Alternatives are ordered by 64-bit keys (value, then lower id first), all distinct. Whenever a thread's 16 elements reach a
// floor, their place and maximum are listed; the floor is the n_top-th largest of the running maxima of 64 groups of threads: n_top
// elements reach it, so no alternative is left out. It is first taken over the first stage alone and then raised by one
// warp a stage in turn, without a barrier: a maximum that another warp has not yet written only leaves the floor lower. About
// 24 (ln stages + 2) places are listed at n_top = 20. At the end the places that reach the last floor are read again, their
// elements that reach it are listed, and a key's place is the number of larger keys. A list that does not fit (many
// equal elements, or rows that rise towards their end) is given up: the threads whose own maximum
// reaches the floor have all their elements read again, each warp keeps its best 32 and these are merged.
// (512 bf16 rows of 151,936, n_top 20: reading all elements of the owning threads again costs 12 to 20 us of 55, listing single
// elements as they pass 28.)
// Bound: for many rows the slots of the SMs whose last row runs alone (512 rows, 3.4 an SM, take 47 us, half of the copy rate of HBM; 608, four an
// SM, 48 us; 2,048 138 us, 68%, with two stages a CTA, 167 us with one) and their issue slots, 60% used; a dependent chain of
// loads, cluster joins and places for a few (8 f32 rows: 11 us).
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "tc_device.cuh"

namespace dlite {
namespace {

constexpr int kGroups = 64;  // groups of threads behind the floor
constexpr int kList = 512;   // listed places, and listed elements, at most
constexpr int kMaxCluster = 8;

struct LpArgs {
  int V, n_top;
  long long stride;
  const void* x;
  const int32_t* tok;
  float T, k;  // k = log2(e) / T
  float *lp, *ent;
  int32_t* ids;
  float* top;
  int* status;
};

// Softmax statistics of a set of elements: the largest, how often it occurs, and over the
// others s = sum 2^(-d k), w = sum 2^(-d k) d with d = m - x.
struct Stat {
  float m, n, s, w;
};
// Weight of a distance d >= 0; one beyond 2^-200 is 0, and its d (perhaps infinite) is taken as 0.
__device__ __forceinline__ float weight(float& d, float k) {
  const float e = d * k;
  if (e > 200.f) {
    d = 0.f;
    return 0.f;
  }
  return tc::ex2_approx(-e);
}
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, float k) {
  const bool up = b.m > a.m;
  const Stat hi = up ? b : a, lo = up ? a : b;
  if (lo.m == hi.m) return {hi.m, hi.n + lo.n, hi.s + lo.s, hi.w + lo.w};
  // lo.n = 0 and lo.s = 0 (no element, or only -inf): nothing to take along. A NaN sum stays.
  float d = hi.m - lo.m;
  const float f = weight(d, k), t = lo.n + lo.s;
  return {hi.m, hi.n, hi.s + f * t, hi.w + f * (lo.w + d * t)};
}

// The statistics of a warp's lanes together, the same bits in every lane
__device__ __forceinline__ Stat warp_join(Stat v, float k, int lane) {
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
    const Stat b = {__shfl_xor_sync(0xffffffffu, v.m, o), __shfl_xor_sync(0xffffffffu, v.n, o),
                    __shfl_xor_sync(0xffffffffu, v.s, o), __shfl_xor_sync(0xffffffffu, v.w, o)};
    const bool up = lane & o;  // the same order of the two on both lanes
    v = join(up ? b : v, up ? v : b, k);
  }
  return v;
}

// Order of the alternatives: larger logit first (-0 = +0, NaN as -inf), then the lower id; 0 = no element.
__device__ __forceinline__ uint64_t key_of(float x, int id) {
  x = x != x ? -INFINITY : x + 0.f;
  uint32_t u = __float_as_uint(x);
  u = u & 0x80000000u ? ~u : u | 0x80000000u;
  return ((uint64_t)u << 32) | (uint32_t)~id;
}
__device__ __forceinline__ int id_of(uint64_t key) { return (int)~(uint32_t)key; }
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int src) { return __shfl_sync(0xffffffffu, v, src); }
__device__ __forceinline__ uint64_t shfl64_xor(uint64_t v, int mask) { return __shfl_xor_sync(0xffffffffu, v, mask); }

// Warp-wide sort of one key per lane, largest in lane 0 (bitonic).
__device__ __forceinline__ uint64_t warp_sort_desc(uint64_t v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int j = size >> 1; j > 0; j >>= 1) {
      const uint64_t o = shfl64_xor(v, j);
      const bool desc = (lane & size) == 0, first = (lane & j) == 0;
      const bool take_max = desc == first;
      v = take_max ? (v > o ? v : o) : (v > o ? o : v);
    }
  return v;
}
// The 32 largest of two descending lists (one key per lane each), descending.
__device__ __forceinline__ uint64_t warp_merge_desc(uint64_t a, uint64_t b, int lane) {
  const uint64_t r = shfl64(b, 31 - lane);
  uint64_t v = a > r ? a : r;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    const uint64_t o = shfl64_xor(v, j);
    v = (lane & j) == 0 ? (v > o ? v : o) : (v > o ? o : v);
  }
  return v;
}
// One warp: the 32 largest of `lists` descending lists of 32 keys.
__device__ __forceinline__ uint64_t warp_merge_lists(const uint64_t* keys, int lists, int lane) {
  uint64_t best = keys[lane];
  for (int i = 1; i < lists; ++i) best = warp_merge_desc(best, keys[32 * i + lane], lane);
  return best;
}

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// The elements of a 16-byte piece as float
template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, float* v) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __uint_as_float(u[i]);
    } else {
      v[2 * i] = lo_f32(u[i]);
      v[2 * i + 1] = hi_f32(u[i]);
    }
  }
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A list of keys of a CTA
struct Top {
  bool on;
  float floor;
  uint64_t* list;
  int* n;
  __device__ __forceinline__ void add(float v, int id) const {
    if (*(volatile int*)n > kList) return;  // given up
    const int at = atomicAdd(n, 1);
    if (at < kList) list[at] = key_of(v, id);
  }
};

constexpr float kTame = 1.2676506002282294e30f;  // 2^100
constexpr uint32_t kFloorBf16x2 = 0xF200F200u;   // -2^101, twice

// out[i] = the i-th largest of n distinct keys, i < n_top (the block's threads, no barrier here)
template <int NT>
__device__ __forceinline__ void place(const uint64_t* keys, int n, int n_top, uint64_t* out) {
  for (int i = threadIdx.x; i < n; i += NT) {
    const uint64_t key = keys[i];
    int above = 0;
    for (int j = 0; j < n; ++j) above += keys[j] > key;
    if (above < n_top) out[above] = key;
  }
}

// The n-th largest (from 1) of 64 values, by one warp (bitonic sort of two a lane).
__device__ __forceinline__ float nth_largest64(const volatile float* g, int n, int lane) {
  float v[2] = {g[lane], g[32 + lane]};
#pragma unroll
  for (int size = 2; size <= 64; size <<= 1)
#pragma unroll
    for (int j = size >> 1; j > 0; j >>= 1) {
      if (j == 32) {
        const float hi = fmaxf(v[0], v[1]), lo = fminf(v[0], v[1]);
        v[0] = hi, v[1] = lo;
      } else {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float o = __shfl_xor_sync(0xffffffffu, v[r], j);
          const bool desc = size == 64 || (size == 32 ? r == 0 : (lane & size) == 0);
          v[r] = ((lane & j) == 0) == desc ? fmaxf(v[r], o) : fminf(v[r], o);
        }
      }
    }
  const float a = __shfl_sync(0xffffffffu, v[0], (n - 1) & 31), b = __shfl_sync(0xffffffffu, v[1], (n - 1) & 31);
  return n <= 32 ? a : b;
}

// The largest of N words of elements of type T (NaN ignored)
template <typename T, int N>
__device__ __forceinline__ float max_of(const uint32_t (&x)[N]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t c = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) c = max_bf16x2(c, x[i]);
    return fmaxf(lo_f32(c), hi_f32(c));
  } else {
    float c = __uint_as_float(x[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) c = fmaxf(c, __uint_as_float(x[i]));
    return c;
  }
}

// One warp takes N words a lane of elements of type T (-inf where a lane has fewer). st.m is the
// warp's running maximum, the same in every lane; own: the lane's largest element.
// The usual step, all elements below a maximum of moderate size, runs two elements an
// instruction: elements below -2^101 (excluded ones: -inf, the type's lowest) become
// -2^101, whose weight is 0 too and whose distance stays finite.
// Elements whose maximum reaches the floor of `top` go to its list, as the place id0 of the first.
template <typename T, int N>
__device__ __forceinline__ void take(const uint32_t (&x)[N], int id0, bool real, float k, Stat& st, float& own,
                                     const Top& top) {
  constexpr int E = sizeof(T) == 4 ? 1 : 2;
  const float cm = max_of<T>(x);
  own = fmaxf(own, cm);
  if (top.on && real && (cm >= top.floor || top.floor == -INFINITY)) top.add(cm, id0);
  const float wm = warp_max_f32(cm);
  if (wm < st.m && fabsf(st.m) < kTame && k > 1e-20f && N * E % 2 == 0) {
    const uint64_t m2 = pack2f(st.m, st.m), k2 = pack2f(-k, -k);
    uint64_t s2 = 0, w2 = 0;
#pragma unroll
    for (int i = 0; i < N * E / 2; ++i) {
      uint64_t v;
      if constexpr (E == 2) {
        const uint32_t c = max_nan_bf16x2(x[i], kFloorBf16x2);
        v = pack2f(lo_f32(c), hi_f32(c));
      } else {
        v = pack2f(max_nan(__uint_as_float(x[2 * i]), -2.f * kTame), max_nan(__uint_as_float(x[2 * i + 1]), -2.f * kTame));
      }
      const uint64_t d = sub2(m2, v), t = mul2(d, k2);
      const uint64_t e = pack2f(tc::ex2_approx(lo2f(t)), tc::ex2_approx(hi2f(t)));
      s2 = add2(s2, e);
      w2 = fma2(e, d, w2);
    }
    st.s += lo2f(s2) + hi2f(s2);
    st.w += lo2f(w2) + hi2f(w2);
    return;
  }
  if (wm > st.m) {
    const float t = st.n + st.s;
    float d = wm - st.m;
    const float f = weight(d, k);   // nothing yet (m = -inf): 0
    st.w = f * (st.w + d * t);
    st.s = f * t;
    st.n = 0.f;
    st.m = wm;
  }
#pragma unroll
  for (int i = 0; i < N * E; ++i) {
    const float v = E == 2 ? (i & 1 ? hi_f32(x[i / 2]) : lo_f32(x[i / 2])) : __uint_as_float(x[i]);
    // no branches: the maximum itself is counted, an element too far below it (or -inf) is nothing, a NaN stays
    const bool top = v == st.m;
    const float d = st.m - v, t = d * k;
    const bool none = top || t > 200.f;
    const float e = none ? 0.f : tc::ex2_approx(-t);
    st.n += top && v > -INFINITY ? 1.f : 0.f;
    st.s += e;
    st.w = fmaf(e, none ? 0.f : d, st.w);
  }
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Store to the same shared-memory variable of CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster_u64(uint64_t* local, uint32_t rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(tc::map_to_rank(tc::su32(local), rank)), "l"(v) : "memory");
}

// Stages of four pieces a thread; their number is the launch's.
template <int NT>
struct Ring {
  static constexpr int PIECES = 4 * NT, BYTES = PIECES * 16, MAX_STAGES = 8;
};

// The kernel's shared memory but for the ring
template <int NT>
struct Shared {
  uint64_t full[Ring<NT>::MAX_STAGES], empty[Ring<NT>::MAX_STAGES];
  uint64_t list[kList], cand[kList];  // places, and elements, that reach the floor
  uint64_t result[32];                // this CTA's alternatives
  // of rank 0: what the CTAs of the cluster send
  uint64_t gather_key[kMaxCluster * 32];
  Stat gather_stat[kMaxCluster];
  Stat stats[NT / 32];
  float group_max[kGroups];
  uint16_t owner[NT];
  int n_owner, n_list, n_cand;
  float s_floor, s_ref;
};
constexpr int kSmSmem = 228 * 1024, kCtaSmem = 227 * 1024;  // of an SM, of which a resident CTA takes 1 KB for itself; at most of a CTA
constexpr int kMostCtas = 5;                                // an SM
// Dynamic shared memory of a CTA when `res` are to be resident
template <int NT>
constexpr int dynamic_smem(int res) {
  constexpr int own = (int)(sizeof(Shared<NT>) + 127) / 128 * 128;
  const int left = kSmSmem / res - 1024 - own, most = kCtaSmem - own;
  return (left < most ? left : most) / 1024 * 1024;
}
static_assert(dynamic_smem<256>(kMostCtas) >= 2 * Ring<256>::BYTES, "copies are under way while a stage is read");

template <typename T, int NT>
__global__ void __launch_bounds__(NT) token_logprobs_kernel(LpArgs a, int C, int stages) {
  using R = Ring<NT>;
  constexpr int E = 16 / sizeof(T), NW = NT / 32, GS = NT / kGroups;
  extern __shared__ __align__(128) uint8_t ring[];
  static_assert(kList >= NT, "the merges' lists share the list's memory");
  __shared__ __align__(16) Shared<NT> sh;
  auto& full = sh.full; auto& empty = sh.empty; auto& list = sh.list; auto& cand = sh.cand; auto& result = sh.result;
  auto& gather_key = sh.gather_key; auto& gather_stat = sh.gather_stat; auto& stats = sh.stats;
  auto& group_max = sh.group_max; auto& owner = sh.owner;
  int &n_owner = sh.n_owner, &n_list = sh.n_list, &n_cand = sh.n_cand;
  float &s_floor = sh.s_floor, &s_ref = sh.s_ref;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / C, rank = C > 1 ? (int)tc::cluster_rank() : 0;
  const int tok = a.tok[row];
  if (tok < 0) {  // not scored: the whole cluster leaves
    if (rank == 0) {
      if (tid == 0 && a.lp) a.lp[row] = 0.f;
      if (tid == 0 && a.ent) a.ent[row] = 0.f;
      if (tid < a.n_top) {
        a.ids[(size_t)row * a.n_top + tid] = -1;
        a.top[(size_t)row * a.n_top + tid] = 0.f;
      }
    }
    return;
  }
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // waited for before the first remote store
  const T* x = static_cast<const T*>(a.x) + row * a.stride;
  // elements before the first 16-byte border, whole pieces, the rest
  const int head = min(a.V, (int)(((16 - ((uintptr_t)x & 15)) & 15) / sizeof(T)));
  const int nv = (a.V - head) / E, tail = head + nv * E;
  const int v0 = (int)((long long)nv * rank / C), v1 = (int)((long long)nv * (rank + 1) / C);
  const uint4* body = reinterpret_cast<const uint4*>(x + head);

  if (tid < 32) result[tid] = 0;
  if (tid < kGroups) group_max[tid] = -INFINITY;
  if (tid == 0) {
    n_list = n_cand = n_owner = 0;
    s_floor = -INFINITY;  // stays where fewer than n_top groups hold elements
    for (int i = 0; i < stages; ++i) {
      tc::mbar_init(tc::su32(full + i), 1);
      tc::mbar_init(tc::su32(empty + i), NW);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  auto issue = [&](int c, int st) {  // thread 0: chunk c of the slice into stage st
    const uint32_t bar = tc::su32(full + st), bytes = 16 * min(R::PIECES, v1 - v0 - c * R::PIECES);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc::mbar_expect_tx(bar, bytes);
    tc::bulk_load(tc::su32(ring + st * R::BYTES), body + v0 + c * R::PIECES, bytes, bar);
  };
  if (tid == 0)
    for (int c = 0; c < stages && v0 + c * R::PIECES < v1; ++c) issue(c, c);

  T x_tok = T(0.f);
  if (tid == NT - 1 && tok < a.V) x_tok = x[tok];  // early: its latency passes under the row's
  const int chunks = (v1 - v0 + R::PIECES - 1) / R::PIECES;
  const int first = tid & ~31;  // the warp's first thread: all loops are the warp's
  bool ok = true;
  float ref = -INFINITY;
  Top top = {a.n_top > 0, -INFINITY, list, &n_list};
  if (chunks) {
    // the first stage alone: its maximum is every warp's first reference (later rescales are rare then), the
    // maxima of groups of threads give the first floor
    ok = tc::mbar_wait_hint(tc::su32(full), 0, a.status);
    float cm = -INFINITY;
    const int n = ok ? min(R::PIECES, v1 - v0) : 0;
    for (int q = tid; q < n; q += NT) {
      uint32_t v[4];
      *reinterpret_cast<uint4*>(v) = reinterpret_cast<const uint4*>(ring)[q];
      cm = fmaxf(cm, max_of<T>(v));
    }
#pragma unroll
    for (int o = GS / 2; o > 0; o >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, o));
    if (tid % GS == 0) group_max[tid / GS] = cm;
    __syncthreads();
    if (warp == 0) {
      const float g = warp_max_f32(fmaxf(group_max[lane], group_max[32 + lane]));
      const float f = a.n_top ? nth_largest64(group_max, a.n_top, lane) : 0.f;
      if (lane == 0) {
        s_ref = g;
        s_floor = f;
      }
    }
    __syncthreads();
    ref = s_ref;
    top.floor = s_floor;
  }

  Stat st = {ref, 0.f, 0.f, 0.f};
  float own = -INFINITY;
  auto group_maxima = [&](float v) {
#pragma unroll
    for (int o = GS / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    // the first stage's maxima, of the same threads' elements, stand until these reach them
    if (tid % GS == 0) *(volatile float*)&group_max[tid / GS] = fmaxf(v, *(volatile float*)&group_max[tid / GS]);
  };
  if (rank == 0 && first < head) {
    const uint32_t v[1] = {__float_as_uint(tid < head ? to_f32(x[tid]) : -INFINITY)};
    take<float>(v, tid, tid < head, a.k, st, own, top);
  }
  constexpr int P = sizeof(T) == 4 ? 4 : 2;  // pieces taken at once: 16 elements
  int stage = 0;
  uint32_t phase = 0;  // of the stage's turn
  for (int c = 0; c < chunks; ++c) {
    // the stage of chunk c - 1 is refilled now: the other warps have had a chunk's time to leave it
    if (tid == 0 && c >= 1 && c - 1 + stages < chunks) {
      ok &= tc::mbar_wait_hint(tc::su32(empty + (stage ? stage : stages) - 1), stage ? phase : phase ^ 1u, a.status);
      if (ok) issue(c - 1 + stages, (stage ? stage : stages) - 1);
    }
    ok = ok && tc::mbar_wait_hint(tc::su32(full + stage), phase, a.status);
    // a copy never landed: the status says so, the row's outputs mean nothing; the barriers below are kept
    const int n = __all_sync(0xffffffffu, ok) ? min(R::PIECES, v1 - v0 - c * R::PIECES) : 0;
    const uint4* src = reinterpret_cast<const uint4*>(ring + stage * R::BYTES);
    if (n == R::PIECES) {
#pragma unroll
      for (int u = 0; u < 4; u += P) {
        uint32_t v[4 * P];
#pragma unroll
        for (int q = 0; q < P; ++q) *reinterpret_cast<uint4*>(v + 4 * q) = src[tid + (u + q) * NT];
        take<T>(v, head + (v0 + c * R::PIECES + tid + u * NT) * E, true, a.k, st, own, top);
      }
    } else {
      constexpr uint32_t none = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;  // -inf
      for (int q = tid, qw = first; qw < n; q += NT, qw += NT) {
        uint32_t v[4];
        *reinterpret_cast<uint4*>(v) = q < n ? src[q] : make_uint4(none, none, none, none);
        take<T>(v, head + (v0 + c * R::PIECES + q) * E, q < n, a.k, st, own, top);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(tc::su32(empty + stage));
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
    if (a.n_top) {
      group_maxima(own);
      if (c % NW == warp) {
        const float f = nth_largest64(group_max, a.n_top, lane);
        if (lane == 0 && f > *(volatile float*)&s_floor) *(volatile float*)&s_floor = f;  // lower ones are floors too
      }
      top.floor = fmaxf(top.floor, *(volatile float*)&s_floor);
    }
  }
  if (tid == 0 && !ok)  // let the copies in flight end (bounded) before the memory is given back
    for (int i = 0; i < stages && i < chunks; ++i)
      for (uint32_t ph = 0; ph < 2; ++ph) tc::mbar_wait_hint(tc::su32(full + i), ph, a.status);
  if (rank == C - 1 && tail + first < a.V) {
    const uint32_t v[1] = {__float_as_uint(tail + tid < a.V ? to_f32(x[tail + tid]) : -INFINITY)};
    take<float>(v, tail + tid, tail + tid < a.V, a.k, st, own, top);
  }

  const Stat all = warp_join(st, a.k, lane);
  if (lane == 0) stats[warp] = all;
  if (a.n_top) group_maxima(own);
  __syncthreads();
  if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // rank 0 runs
  if (warp == NW - 1) {  // the last warp joins the warps' statistics while the others look for alternatives
    Stat b = lane < NW ? stats[lane] : Stat{-INFINITY, 0.f, 0.f, 0.f};
    b = warp_join(b, a.k, lane);
    if (C > 1) {
      if (lane < 2) {
        const uint64_t v = lane ? ((uint64_t)__float_as_uint(b.w) << 32) | __float_as_uint(b.s)
                                : ((uint64_t)__float_as_uint(b.n) << 32) | __float_as_uint(b.m);
        st_cluster_u64(reinterpret_cast<uint64_t*>(&gather_stat[rank]) + lane, 0, v);
      }
    } else if (lane == 0) {
      gather_stat[0] = b;
    }
  }
  if (a.n_top) {
    // the last floor, and the elements of the places that reach it
    top.floor = nth_largest64(group_max, a.n_top, lane);
    const int places = n_list;
    if (places <= kList) {
      const Top found = {true, top.floor, cand, &n_cand};
      auto offer = [&](float v, int id) {
        if (v >= found.floor || found.floor == -INFINITY) found.add(v, id);
      };
      for (int i = tid; i < places * P; i += NT) {
        const uint64_t key = list[i / P];
        if (value_of(key) < top.floor) continue;
        const int id = id_of(key), u = i % P;
        if (id < head || id >= tail) {
          if (u == 0) offer(to_f32(x[id]), id);
          continue;
        }
        const int q = (id - head) / E, chunk = (q - v0) / R::PIECES;
        const bool whole = (chunk + 1) * R::PIECES <= v1 - v0;  // taken P pieces at a time, NT apart
        if (u && !whole) continue;
        float v[E];
        unpack<T>(body[q + u * NT], v);
#pragma unroll
        for (int e = 0; e < E; ++e) offer(v[e], id + u * NT * E + e);
      }
      __syncthreads();
    }
    if (places <= kList && n_cand <= kList) {
      place<NT>(cand, n_cand, a.n_top, result);
    } else {  // too many: each warp keeps the best 32 of its owners' elements, and the warps' lists are merged
      if (!(own < top.floor)) owner[atomicAdd(&n_owner, 1)] = (uint16_t)tid;
      __syncthreads();
      uint64_t best = 0;
      auto batch = [&](uint64_t key) {
        if (!__any_sync(0xffffffffu, key > shfl64(best, 31))) return;
        best = warp_merge_desc(best, warp_sort_desc(key, lane), lane);
      };
      for (int o = warp; o < n_owner; o += NW) {
        const int t = owner[o];
        if (rank == 0 && t < head) batch(lane == 0 ? key_of(to_f32(x[t]), t) : 0);
        if (rank == C - 1 && tail + t < a.V) batch(lane == 0 ? key_of(to_f32(x[tail + t]), tail + t) : 0);
        for (int q0 = v0 + t; q0 < v1; q0 += 32 * NT) {
          const int q = q0 + lane * NT;
          float v[E];
          if (q < v1) unpack<T>(body[q], v);
#pragma unroll
          for (int e = 0; e < E; ++e) batch(q < v1 ? key_of(v[e], head + q * E + e) : 0);
        }
      }
      __syncthreads();  // every thread has seen n_list
      list[tid] = best;
      __syncthreads();
      if (warp == 0) result[lane] = warp_merge_lists(list, NW, lane);
    }
  }
  __syncthreads();
  if (warp == 0 && C > 1 && a.n_top) st_cluster_u64(&gather_key[rank * 32 + lane], 0, result[lane]);
  if (C > 1) {
    tc::cluster_sync_all();
    if (rank) return;  // nothing reads this CTA's memory
  } else {
    __syncthreads();
  }
  const Stat all_st = C > 1 ? warp_join(lane < C ? gather_stat[lane] : Stat{-INFINITY, 0.f, 0.f, 0.f}, a.k, lane) : gather_stat[0];
  // a row of -inf alone: every token impossible; +inf or NaN: no distribution
  const bool none = all_st.n == 0.f && all_st.s == 0.f, bad = all_st.m == INFINITY || all_st.s != all_st.s;
  const float logS = bad ? NAN : log1pf(all_st.s + (all_st.n - 1.f));
  auto ln_p = [&](float xv) { return none || (xv == -INFINITY && !bad) ? -INFINITY : -((all_st.m - xv) / a.T) - logS; };
  if (tid == NT - 1) {
    if (a.lp) a.lp[row] = tok < a.V ? ln_p(to_f32(x_tok)) : NAN;
    if (tok >= a.V) flag_status(a.status, kDevBounds);
    if (a.ent) a.ent[row] = none ? 0.f : logS + all_st.w / a.T / (all_st.n + all_st.s);
  }
  if (tid < (a.n_top ? 32 * C : 0) && lane < a.n_top) {
    const uint64_t key = C > 1 ? gather_key[tid] : result[lane];
    int above = C > 1 ? 0 : lane;
    for (int c = 0; c < C && C > 1 && above < a.n_top; ++c)  // descending lists
      for (int i = 0; i < a.n_top && above < a.n_top && gather_key[c * 32 + i] > key; ++i) ++above;
    if (key && above < a.n_top) {
      a.ids[(size_t)row * a.n_top + above] = id_of(key);
      a.top[(size_t)row * a.n_top + above] = ln_p(value_of(key));
    }
  }
}

}  // namespace
}  // namespace dlite

extern "C" int dlite_token_logprobs(const dlite_logprobs_args* g, dlite_stream_t stream) {
  using namespace dlite;
  if (!g || !g->logits || !g->tokens) return DLITE_ERR_INVALID_ARG;
  if (g->rows < 1 || g->V < 1 || g->stride < g->V || g->n_top < 0 || g->n_top > g->V) return DLITE_ERR_INVALID_ARG;
  if (g->dtype != DLITE_F32 && g->dtype != DLITE_BF16) return DLITE_ERR_INVALID_ARG;
  if (!(g->temperature > 0.f) || isinf(g->temperature)) return DLITE_ERR_INVALID_ARG;
  if (g->n_top && (!g->top_ids || !g->top_logprobs)) return DLITE_ERR_INVALID_ARG;
  if ((uintptr_t)g->logits % (g->dtype == DLITE_F32 ? 4 : 2) ||
      !aligned4(g->tokens, g->logprob, g->entropy, g->top_ids, g->top_logprobs, g->status))
    return DLITE_ERR_INVALID_ARG;
  if (g->n_top > DLITE_MAX_TOP || g->rows > (1 << 27) || g->V > (1 << 30)) return DLITE_ERR_UNSUPPORTED_SHAPE;
  LpArgs a = {};
  a.V = g->V;
  a.n_top = g->n_top;
  a.stride = g->stride;
  a.x = g->logits;
  a.tok = g->tokens;
  a.T = g->temperature;
  a.k = (float)(1.4426950408889634 / (double)g->temperature);
  a.lp = g->logprob;
  a.ent = g->entropy;
  a.ids = g->top_ids;
  a.top = g->top_logprobs;
  a.status = g->status;
  // Rows are split among a cluster until there are two CTAs an SM, as long as a slice keeps two stages; CTAs of 512
  // threads where even then an SM has only one. (bf16 rows of 151,936, n_top 20: 64 rows 17.0 us with one CTA an SM, 19.3 with
  // two; 200 rows 32.9, 28.8, and 38.7 with three: what a CTA does apart from reading takes about 6 us.)
  const int es = g->dtype == DLITE_F32 ? 4 : 2;
  int C = 1;
  while (C < kMaxCluster && (long long)C * g->rows < 2LL * device_sms() && (long long)g->V * es >= 4LL * C * Ring<256>::BYTES) C *= 2;
  const bool wide = (long long)C * g->rows <= device_sms();
  void (*fn)(LpArgs, int, int) = g->dtype == DLITE_F32 ? (wide ? token_logprobs_kernel<float, 512> : token_logprobs_kernel<float, 256>)
                                                       : (wide ? token_logprobs_kernel<bf16, 512> : token_logprobs_kernel<bf16, 256>);
  // Residency: as many CTAs an SM as the rows come to (at most 5), no more: with room for more the rows are spread unevenly
  // (456 rows, three an SM, took as long as 608). What shared memory that leaves holds stages.
  const int res = (int)std::min<long long>(kMostCtas, std::max(1LL, ((long long)C * g->rows + device_sms() - 1) / device_sms()));
  const int smem = wide ? dynamic_smem<512>(res) : dynamic_smem<256>(res);
  const int stages = std::min(smem / (wide ? Ring<512>::BYTES : Ring<256>::BYTES), (int)Ring<256>::MAX_STAGES);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C * g->rows);
  cfg.blockDim = dim3(wide ? 512 : 256);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = C;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = C > 1 ? 2 : 1;
  // always the same: the attribute is the process's, and another thread may launch between the two calls
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       wide ? dynamic_smem<512>(1) : dynamic_smem<256>(1));
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, fn, a, C, stages);
  return launch_status(e);
}
