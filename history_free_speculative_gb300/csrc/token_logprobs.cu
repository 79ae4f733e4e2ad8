// Log probabilities of given tokens, entropy and the top alternatives of rows of
// logits, in one pass over the row.
//
// With m the row's largest logit and d_v = (m - x_v) / T >= 0: S = sum e^-d, log p(v) = -d_v - log S,
// H = log S + (sum e^-d d) / S; every term is >= 0, so nothing cancels. The largest
// elements' own ones are counted apart (n) from the other terms (s), and log S = log1p(s + n - 1):
// a row that is nearly certain keeps its small entropy to full precision.
//
// A row is read by a cluster of CTAs (one when there are many rows), each a slice, each thread
// every blockDim-th 16-byte piece of the slice, in four pieces in flight. A thread keeps
// (m, n, s, w = sum e^-d d) online and the place of its largest element. The thread maxima,
// as 64-bit keys (value, then lower id first, all distinct), give the alternatives: at most n_top
// threads can own one, namely those with the n_top largest keys, and an alternative is never below
// the n_top-th of those keys. Each warp takes some of those threads, reads their elements
// again (L2) and keeps the best 32 across its lanes; a tournament over the warps, then one over the CTAs, ends it.
// Bound: HBM for many rows, a dependent chain of a few microseconds for a few.
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "tc_device.cuh"

namespace dlite {
namespace {

constexpr int kMaxTop = DLITE_MAX_TOP;
constexpr int kThreads = 512;
constexpr int kNW = kThreads / 32;
constexpr float kLn2 = 0.6931471805599453f;

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
// others s = sum 2^-d, w = sum 2^-d d with d = (m - x) k.
struct Stat {
  float m, n, s, w;
};
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, float k) {
  const bool up = b.m > a.m;
  const Stat hi = up ? b : a, lo = up ? a : b;
  if (lo.m == hi.m) return {hi.m, hi.n + lo.n, hi.s + lo.s, hi.w + lo.w};
  // lo.n = 0 and lo.s = 0 (no element, or only -inf): nothing to take along. A NaN sum stays.
  const float d = fminf((hi.m - lo.m) * k, 1e4f), f = tc::ex2_approx(-d), t = lo.n + lo.s;
  return {hi.m, hi.n, hi.s + f * t, hi.w + f * (lo.w + d * t)};
}

// Order of the alternatives: larger logit first (-0 = +0, NaN as -inf), then the lower id; 0 = no element.
__device__ __forceinline__ uint64_t key_of(float x, int id) {
  x = x != x ? -INFINITY : x + 0.f;
  uint32_t u = __float_as_uint(x);
  u = u & 0x80000000u ? ~u : u | 0x80000000u;
  return ((uint64_t)u << 32) | (uint32_t)~id;
}
__device__ __forceinline__ int id_of(uint64_t key) { return (int)~(uint32_t)key; }

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

// E elements of type T at p as float: one 16-byte access
template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, float* v) {
  if constexpr (sizeof(T) == 4) {
    v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
  } else {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}

// Takes N elements with ids id0 .. id0 + N - 1 into the statistics; idx: id of the first largest.
template <int N>
__device__ __forceinline__ void take(const float (&v)[N], int id0, float k, Stat& st, int& idx) {
  float cm = v[0], cn = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) {
    cm = fmaxf(cm, v[i]);
    cn = fminf(cn, v[i]);
  }
  if (cm > st.m) {
    const float t = st.n + st.s;
    if (st.m == -INFINITY) {
      st.w = st.w + 0.f * t;  // no weight so far; a NaN stays one
      st.s = 0.f * t;
    } else {
      const float d = fminf((cm - st.m) * k, 1e4f), f = tc::ex2_approx(-d);
      st.w = f * (st.w + d * t);
      st.s = f * t;
    }
    st.n = 0.f;
    st.m = cm;
#pragma unroll
    for (int i = N - 1; i >= 0; --i)
      if (v[i] == cm) idx = id0 + i;
  }
  if (cm >= st.m || cn == -INFINITY) {  // the largest is among them, or an excluded id
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (v[i] == -INFINITY) continue;
      if (v[i] == st.m) {
        st.n += 1.f;
        continue;
      }
      const float d = (st.m - v[i]) * k;
      const float e = tc::ex2_approx(-d);
      st.s += e;
      st.w += e * fminf(d, 1e30f);  // d may overflow where e = 0
    }
  } else {
    float s = 0.f, w = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float d = (st.m - v[i]) * k, e = tc::ex2_approx(-d);
      s += e;
      w = fmaf(e, fminf(d, 1e30f), w);
    }
    st.s += s;
    st.w += w;
  }
}

__device__ __forceinline__ uint64_t ld_cluster_u64(const uint64_t* local, uint32_t rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(tc::map_to_rank(tc::su32(local), rank)) : "memory");
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const LpArgs a, int C) {
  constexpr int E = 16 / sizeof(T);
  __shared__ uint64_t lists[kNW * 32];   // sorted keys of the warps
  __shared__ uint64_t result[32];        // this CTA's alternatives
  __shared__ Stat stats[kNW];
  __shared__ __align__(16) Stat cta_stat;
  __shared__ int owners[kMaxTop];
  __shared__ uint64_t s_floor;
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
  const T* x = static_cast<const T*>(a.x) + row * a.stride;
  // elements before the first 16-byte border, whole pieces, the rest
  const int head = min(a.V, (int)(((16 - ((uintptr_t)x & 15)) & 15) / sizeof(T)));
  const int nv = (a.V - head) / E, tail = head + nv * E;
  const int v0 = (int)((long long)nv * rank / C), v1 = (int)((long long)nv * (rank + 1) / C);
  const uint4* body = reinterpret_cast<const uint4*>(x + head);

  Stat st = {-INFINITY, 0.f, 0.f, 0.f};
  int idx = -1;
  auto single = [&](int id) {
    const float v[1] = {to_f32(x[id])};
    if (idx < 0) idx = id;
    take<1>(v, id, a.k, st, idx);
  };
  if (rank == 0 && tid < head) single(tid);
  int p = v0 + tid;
  if (idx < 0 && p < v1) idx = head + p * E;
  for (; p + 3 * kThreads < v1; p += 4 * kThreads) {
    uint4 w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = __ldcs(body + p + u * kThreads);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float v[E];
      unpack<T>(w[u], v);
      take<E>(v, head + (p + u * kThreads) * E, a.k, st, idx);
    }
  }
  for (; p < v1; p += kThreads) {
    float v[E];
    unpack<T>(__ldcs(body + p), v);
    take<E>(v, head + p * E, a.k, st, idx);
  }
  if (rank == C - 1 && tail + tid < a.V) single(tail + tid);

  Stat all = st;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Stat b = {__shfl_xor_sync(0xffffffffu, all.m, o), __shfl_xor_sync(0xffffffffu, all.n, o),
                    __shfl_xor_sync(0xffffffffu, all.s, o), __shfl_xor_sync(0xffffffffu, all.w, o)};
    // the same order of the two on both lanes: bits agree
    all = lane & o ? join(b, all, a.k) : join(all, b, a.k);
  }
  if (lane == 0) stats[warp] = all;

  if (a.n_top) {
    // the n_top threads with the largest keys, and the n_top-th of those keys
    const uint64_t mine = idx < 0 ? 0 : key_of(st.m, idx);
    lists[tid] = warp_sort_desc(mine, lane);
    __syncthreads();
    if (warp == 0) {
      const uint64_t best = warp_merge_lists(lists, kNW, lane);
      const uint64_t fl = shfl64(best, a.n_top - 1);
      if (lane == 0) s_floor = fl ? fl : 1;  // 0: fewer threads with elements than n_top
    }
    if (tid < kMaxTop) owners[tid] = -1;
    __syncthreads();
    const uint64_t floor_key = s_floor;
    // keys are distinct, so a thread's place among the winners is its key's rank
    if (mine >= floor_key) {
      int place = 0;
      for (int w = 0; w < kNW; ++w)
        for (int i = 0; i < a.n_top; ++i) {
          if (lists[w * 32 + i] <= mine) break;
          ++place;
        }
      owners[place] = tid;
    }
    __syncthreads();
    uint64_t best = 0;
    auto batch = [&](uint64_t key) {
      if (key < floor_key) key = 0;
      if (!__any_sync(0xffffffffu, key != 0)) return;
      best = warp_merge_desc(best, warp_sort_desc(key, lane), lane);
    };
    for (int o = warp; o < a.n_top; o += kNW) {
      const int t = owners[o];
      if (t < 0) break;
      if (rank == 0 && t < head) batch(lane == 0 ? key_of(to_f32(x[t]), t) : 0);
      if (rank == C - 1 && tail + t < a.V) batch(lane == 0 ? key_of(to_f32(x[tail + t]), tail + t) : 0);
      for (int q0 = v0 + t; q0 < v1; q0 += 32 * kThreads) {
        const int q = q0 + lane * kThreads;
        float v[E];
        if (q < v1) unpack<T>(body[q], v);
#pragma unroll
        for (int i = 0; i < E; ++i) batch(q < v1 ? key_of(v[i], head + q * E + i) : 0);
      }
    }
    __syncthreads();  // every thread is done with the lists
    lists[tid] = best;
  }
  __syncthreads();
  if (warp == 0) {
    if (a.n_top) result[lane] = warp_merge_lists(lists, kNW, lane);
    Stat b = lane < kNW ? stats[lane] : Stat{-INFINITY, 0.f, 0.f, 0.f};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Stat c = {__shfl_xor_sync(0xffffffffu, b.m, o), __shfl_xor_sync(0xffffffffu, b.n, o),
                      __shfl_xor_sync(0xffffffffu, b.s, o), __shfl_xor_sync(0xffffffffu, b.w, o)};
      b = lane & o ? join(c, b, a.k) : join(b, c, a.k);
    }
    if (lane == 0) cta_stat = b;
  }
  __syncthreads();
  if (C > 1) tc::cluster_sync_all();
  if (rank == 0 && warp == 0) {
    Stat all_st = cta_stat;
    uint64_t best = a.n_top ? result[lane] : 0;
    for (int c = 1; c < C; ++c) {
      const uint64_t* q = reinterpret_cast<const uint64_t*>(&cta_stat);
      const uint64_t lo = ld_cluster_u64(q, c), hi = ld_cluster_u64(q + 1, c);
      all_st = join(all_st, Stat{__uint_as_float((uint32_t)lo), __uint_as_float((uint32_t)(lo >> 32)),
                                 __uint_as_float((uint32_t)hi), __uint_as_float((uint32_t)(hi >> 32))}, a.k);
      if (a.n_top) best = warp_merge_desc(best, ld_cluster_u64(result + lane, c), lane);
    }
    const float S1 = all_st.s + (all_st.n - 1.f);  // S - 1
    // a row of -inf alone: every token impossible; +inf or NaN: no distribution
    const bool none = all_st.n == 0.f && all_st.s == 0.f, bad = all_st.m == INFINITY || all_st.s != all_st.s;
    const float logS = bad ? NAN : log1pf(S1);
    if (lane == 0) {
      if (a.lp) {
        float r = NAN;
        if (tok < a.V) {
          const float xv = to_f32(x[tok]);
          r = none || (xv == -INFINITY && !bad) ? -INFINITY : -((all_st.m - xv) / a.T) - logS;
        } else {
          flag_status(a.status, kDevBounds);
        }
        a.lp[row] = r;
      }
      if (a.ent) a.ent[row] = none ? 0.f : logS + all_st.w * kLn2 / (all_st.n + all_st.s);
    }
    if (lane < a.n_top) {
      const int id = id_of(best);
      const float xv = to_f32(x[id]);
      a.ids[(size_t)row * a.n_top + lane] = id;
      a.top[(size_t)row * a.n_top + lane] = none || (xv == -INFINITY && !bad) ? -INFINITY : -((all_st.m - xv) / a.T) - logS;
    }
  }
  if (C > 1) tc::cluster_sync_all();  // no CTA leaves while another reads its shared memory
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
  if ((uintptr_t)g->logits % (g->dtype == DLITE_F32 ? 4 : 2)) return DLITE_ERR_INVALID_ARG;
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
  // few rows: a cluster per row, so that every SM reads; a slice keeps a piece for every thread
  const int es = g->dtype == DLITE_F32 ? 4 : 2;
  int C = 1;
  while (C < 8 && 2LL * C * g->rows <= 2LL * device_sms() && (long long)g->V * es >= 2LL * C * kThreads * 16) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C * g->rows);
  cfg.blockDim = dim3(kThreads);
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
  return launch_status(g->dtype == DLITE_F32 ? cudaLaunchKernelEx(&cfg, token_logprobs_kernel<float>, a, C)
                                             : cudaLaunchKernelEx(&cfg, token_logprobs_kernel<bf16>, a, C));
}
