// Log probabilities of given tokens, entropy and the top alternatives of rows of
// logits, in one pass over the row.
//
// With m the row's largest logit and d_v = (m - x_v) / T >= 0: S = sum e^-d, log p(v) = -d_v - log S,
// H = log S + (sum e^-d d) / S; every term is >= 0, so nothing cancels. The largest
// elements' own ones are counted apart (n) from the other terms (s), and log S = log1p(s + n - 1):
// a row that is nearly certain keeps its small entropy to full precision.
//
// A row is read by a cluster of CTAs (one when there are many rows), each a slice, each thread
// every blockDim-th 16-byte piece of the slice, four pieces in flight. A warp shares its running maximum m (one
// warp-wide maximum per 16 elements a lane), so that rescaling is a branch the whole warp takes, about ln(steps) times:
// with a maximum per thread some lane of a warp rescaled in most steps (512 bf16 rows of 151,936: 93.5 us). A thread
// keeps (n, s, w = sum e^-d d) and the largest of its own elements.
// Alternatives are ordered by 64-bit keys (value, then lower id first), all distinct. The n_top-th largest of the maxima of 64
// groups of threads is a floor: n_top elements reach it. Only threads whose own maximum reaches the floor can hold an
// alternative; their elements are read again (L2), those that reach the floor are listed, and an
// element's place is the number of larger keys. (64 groups, n_top = 20: about -64 ln(1 - 20 / 64) = 24 elements and
// the floor's equals.) A list that does not fit (many equals, or a thousand large elements in the same few
// threads) is replaced by each warp's best 32, merged.
// Bound: HBM for many rows, a dependent chain of a few microseconds for a few.
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "tc_device.cuh"

namespace dlite {
namespace {

constexpr int kGroups = 64;  // groups of threads behind the floor
constexpr int kList = 1024;  // listed elements
constexpr int kMaxCluster = 8;
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

__device__ __forceinline__ float warp_max_f32(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// One warp takes N elements a lane (-inf where a lane has fewer). st.m is the warp's running
// maximum, the same in every lane; own: the lane's largest element.
template <int N>
__device__ __forceinline__ void take(const float (&v)[N], float k, Stat& st, float& own) {
  float cm = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) cm = fmaxf(cm, v[i]);
  own = fmaxf(own, cm);
  const float wm = warp_max_f32(cm);
  float s = 0.f, w = 0.f;
  if (wm < st.m) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float d = (st.m - v[i]) * k, e = tc::ex2_approx(-d);
      s += e;
      w = fmaf(e, fminf(d, 1e30f), w);  // d = inf, or overflown, where e = 0; a NaN e stays
    }
  } else {  // the largest so far is among them
    if (wm > st.m) {
      const float t = st.n + st.s;
      if (st.m == -INFINITY) {
        st.w = st.w + 0.f * t;  // no weight so far; a NaN stays one
        st.s = 0.f * t;
      } else {
        const float d = fminf((wm - st.m) * k, 1e4f), f = tc::ex2_approx(-d);
        st.w = f * (st.w + d * t);
        st.s = f * t;
      }
      st.n = 0.f;
      st.m = wm;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool top = v[i] == st.m;
      const float d = (st.m - v[i]) * k, e = top ? 0.f : tc::ex2_approx(-d);
      s += e;
      w = fmaf(e, fminf(d, 1e30f), w);
      st.n += top && st.m > -INFINITY ? 1.f : 0.f;
    }
  }
  st.s += s;
  st.w += w;
}

// Store to the same shared-memory variable of CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster_u64(uint64_t* local, uint32_t rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(tc::map_to_rank(tc::su32(local), rank)), "l"(v) : "memory");
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT) token_logprobs_kernel(LpArgs a, int C) {
  constexpr int E = 16 / sizeof(T), NW = NT / 32, GS = NT / kGroups;
  static_assert(kList >= NT, "the merges' lists share the list's memory");
  __shared__ uint64_t list[kList];       // elements that reach the floor
  __shared__ float group_max[kGroups];
  __shared__ uint64_t result[32];        // this CTA's alternatives
  __shared__ Stat stats[NW];
  // of rank 0: what the CTAs of the cluster send
  __shared__ uint64_t gather_key[kMaxCluster * 32];
  __shared__ __align__(16) Stat gather_stat[kMaxCluster];
  __shared__ uint16_t owner[NT];
  __shared__ int n_owner, n_list;
  __shared__ float s_floor;
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

  Stat st = {-INFINITY, 0.f, 0.f, 0.f};
  float own = -INFINITY;
  const int first = tid & ~31;  // the warp's first thread: all loops are the warp's
  if (rank == 0 && first < head) {
    const float v[1] = {tid < head ? to_f32(x[tid]) : -INFINITY};
    take<1>(v, a.k, st, own);
  }
  constexpr int P = 16 / E;  // pieces taken at once: 16 elements
  int p = v0 + tid, pw = v0 + first;
  for (; pw + 31 + 3 * NT < v1; p += 4 * NT, pw += 4 * NT) {
    uint4 w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = __ldcs(body + p + u * NT);
#pragma unroll
    for (int u = 0; u < 4; u += P) {
      float v[P * E];
#pragma unroll
      for (int q = 0; q < P; ++q) unpack<T>(w[u + q], v + q * E);
      take<P * E>(v, a.k, st, own);
    }
  }
  for (; pw < v1; p += NT, pw += NT) {
    float v[E];
    if (p < v1) {
      unpack<T>(__ldcs(body + p), v);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = -INFINITY;
    }
    take<E>(v, a.k, st, own);
  }
  if (rank == C - 1 && tail + first < a.V) {
    const float v[1] = {tail + tid < a.V ? to_f32(x[tail + tid]) : -INFINITY};
    take<1>(v, a.k, st, own);
  }

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
    float gm = own;
#pragma unroll
    for (int o = GS / 2; o > 0; o >>= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
    if (tid % GS == 0) group_max[tid / GS] = gm;
    if (tid == 0) n_owner = n_list = 0;
    if (tid < 32) result[tid] = 0;
    __syncthreads();
    if (tid < kGroups) {
      const float g = group_max[tid];
      int above = 0, reach = 0;
#pragma unroll 16
      for (int i = 0; i < kGroups; ++i) {
        above += group_max[i] > g;
        reach += group_max[i] >= g;
      }
      if (above < a.n_top && reach >= a.n_top) s_floor = g;  // equal groups write the same
    }
    __syncthreads();
    const float floor = s_floor;
    if (!(own < floor)) owner[atomicAdd(&n_owner, 1)] = (uint16_t)tid;
    __syncthreads();
    // the owners' elements: item = (owner, one of its places; the last two are its head and tail elements)
    const int places = (v1 - v0 + NT - 1) / NT + 2, items = n_owner * places;
    auto offer = [&](float v, int id) {
      if (v < floor || (v != v && floor > -INFINITY)) return;
      const int at = atomicAdd(&n_list, 1);
      if (at < kList) list[at] = key_of(v, id);
    };
    for (int i0 = tid; i0 < items; i0 += 4 * NT) {
      uint4 w[4];
      int q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * NT, o = i / places, t = i < items ? owner[o] : 0, j = i - o * places;
        q[u] = -1;
        if (i >= items) continue;
        if (j < places - 2) {
          q[u] = v0 + t + j * NT;
          if (q[u] < v1)
            w[u] = body[q[u]];
          else
            q[u] = -1;
        } else if (j == places - 2) {
          if (rank == 0 && t < head) offer(to_f32(x[t]), t);
        } else if (rank == C - 1 && tail + t < a.V) {
          offer(to_f32(x[tail + t]), tail + t);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (q[u] < 0) continue;
        float v[E];
        unpack<T>(w[u], v);
#pragma unroll
        for (int e = 0; e < E; ++e) offer(v[e], head + q[u] * E + e);
      }
    }
    __syncthreads();
    if (n_list <= kList) {
      const int n = n_list;
      for (int i = tid; i < n; i += NT) {
        const uint64_t key = list[i];
        int above = 0;
        for (int j = 0; j < n; ++j) above += list[j] > key;
        if (above < a.n_top) result[above] = key;
      }
    } else {  // too many: each warp keeps the best 32 of its owners' elements, and the warps' lists are merged
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
  if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // rank 0 runs
  if (warp == 0) {
    Stat b = lane < NW ? stats[lane] : Stat{-INFINITY, 0.f, 0.f, 0.f};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Stat c = {__shfl_xor_sync(0xffffffffu, b.m, o), __shfl_xor_sync(0xffffffffu, b.n, o),
                      __shfl_xor_sync(0xffffffffu, b.s, o), __shfl_xor_sync(0xffffffffu, b.w, o)};
      b = lane & o ? join(c, b, a.k) : join(b, c, a.k);
    }
    if (C > 1) {
      if (lane < 2) {
        const uint64_t v = lane ? ((uint64_t)__float_as_uint(b.w) << 32) | __float_as_uint(b.s)
                                : ((uint64_t)__float_as_uint(b.n) << 32) | __float_as_uint(b.m);
        st_cluster_u64(reinterpret_cast<uint64_t*>(&gather_stat[rank]) + lane, 0, v);
      }
      if (a.n_top) st_cluster_u64(&gather_key[rank * 32 + lane], 0, result[lane]);
    } else if (lane == 0) {
      gather_stat[0] = b;
    }
  }
  if (C > 1) {
    tc::cluster_sync_all();
    if (rank) return;  // nothing reads this CTA's memory
  } else {
    __syncthreads();
  }
  Stat all_st = gather_stat[0];
  for (int c = 1; c < C; ++c) all_st = join(all_st, gather_stat[c], a.k);
  // a row of -inf alone: every token impossible; +inf or NaN: no distribution
  const bool none = all_st.n == 0.f && all_st.s == 0.f, bad = all_st.m == INFINITY || all_st.s != all_st.s;
  const float logS = bad ? NAN : log1pf(all_st.s + (all_st.n - 1.f));
  auto ln_p = [&](float xv) { return none || (xv == -INFINITY && !bad) ? -INFINITY : -((all_st.m - xv) / a.T) - logS; };
  if (tid == NT - 1) {
    if (a.lp) a.lp[row] = tok < a.V ? ln_p(to_f32(x[tok])) : NAN;
    if (tok >= a.V) flag_status(a.status, kDevBounds);
    if (a.ent) a.ent[row] = none ? 0.f : logS + all_st.w * kLn2 / (all_st.n + all_st.s);
  }
  if (tid < (a.n_top ? 32 * C : 0)) {
    uint64_t key = result[lane];
    int above = lane;
    if (C > 1) {
      key = gather_key[tid];
      above = 0;
      for (int j = 0; j < 32 * C; ++j) above += gather_key[j] > key;
    }
    if (key && above < a.n_top) {
      const int id = id_of(key);
      a.ids[(size_t)row * a.n_top + above] = id;
      a.top[(size_t)row * a.n_top + above] = ln_p(to_f32(x[id]));
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
  // few rows: a cluster per row, so that every SM reads; a slice keeps four pieces for every thread. Many rows:
  // CTAs of 256 threads, of which an SM holds several at different places of their rows.
  const int es = g->dtype == DLITE_F32 ? 4 : 2;
  int C = 1;
  while (C < kMaxCluster && 2LL * C * g->rows <= 2LL * device_sms() && (long long)g->V * es >= 2LL * C * 512 * 16 * 4) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C * g->rows);
  cfg.blockDim = dim3(C > 1 ? 512 : 256);
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
  void (*fn)(LpArgs, int) = g->dtype == DLITE_F32 ? (C > 1 ? token_logprobs_kernel<float, 512> : token_logprobs_kernel<float, 256>)
                                                  : (C > 1 ? token_logprobs_kernel<bf16, 512> : token_logprobs_kernel<bf16, 256>);
  return launch_status(cudaLaunchKernelEx(&cfg, fn, a, C));
}
