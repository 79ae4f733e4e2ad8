// Rotary positions of the target side: the table of (cos, sin) and its
// application to heads of queries (the keys of the paged cache are rotated on
// their way in, kv_cache.cu, by the same arithmetic).
//
// rope_kernel: one block per token. A head's columns are cut into items of V
// columns (16 bytes): V / 2 neighbouring pairs (interleaved), V columns of the
// first half with their V partners (half), or V columns past the rotated part.
// Thread u of the block takes items u, u + blockDim, ... of the token's heads;
// lanes next to each other hold neighbouring items, so a warp's loads are
// contiguous. Bound: HBM (each element once in, once out) for prompts (80% of the copy
// rate for a float32 prompt of 268 MB in and out, 50.5 us); launch and one dependent load (position -> table -> store) for a
// decoded token (2.0 us in a graph).
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "rope.cuh"

namespace dlite {
namespace {

struct RopeFreq {
  double f[128];
};

__global__ void rope_table_kernel(RopeFreq fr, int half, int n_pos, double m, float2* table) {
  pdl_trigger();
  pdl_wait();
  const long long n = (long long)n_pos * half, stride = (long long)gridDim.x * blockDim.x;
  for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += stride) {
    const int p = (int)(e / half), i = (int)(e % half);
    double s, c;
    sincos((double)p * fr.f[i], &s, &c);
    table[e] = make_float2((float)(m * c), (float)(m * s));
  }
}

struct RopeArgs {
  int T, heads, d_h, half, n_pos, copy;  // copy: the columns past the rotated part are copied
  const void* x;
  long long xs;
  void* out;
  long long os;
  const int64_t* pos;
  const int32_t* n_rows;
  const float2* table;
  int* status;
};

// V consecutive values of T as float, by one 16-byte access (V = 16 / sizeof(T)) or one element (V = 1)
template <typename T, int V>
__device__ __forceinline__ void load_vals(const T* p, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = to_f32(*p);
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = to_f32(e[i]);
  }
}
__device__ __forceinline__ void from_f32(float x, float& y) { y = x; }
__device__ __forceinline__ void from_f32(float x, bf16& y) { y = __float2bfloat16_rn(x); }
template <typename T, int V>
__device__ __forceinline__ void store_vals(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    from_f32(v[0], *p);
  } else {
    uint4 w;
    T* e = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int i = 0; i < V; ++i) from_f32(v[i], e[i]);
    *reinterpret_cast<uint4*>(p) = w;
  }
}

// V: columns per access of the half layout; interleaved items hold V columns = V / 2 pairs (V = 1: one pair)
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(256) rope_kernel(RopeArgs a) {
  pdl_trigger();
  pdl_wait();
  const long long tok = blockIdx.x;
  const int b = (int)(blockIdx.x / (unsigned)a.T), t = (int)(blockIdx.x - (unsigned)b * (unsigned)a.T);
  if (a.n_rows && t >= a.n_rows[b]) return;
  long long p = first_position(a.pos, b) + t;
  if (p < 0 || p >= a.n_pos) {
    if (threadIdx.x == 0) flag_status(a.status, kDevBounds);
    p = p < 0 ? 0 : a.n_pos - 1;
  }
  const float2* tab = a.table + p * a.half;
  const T* x = static_cast<const T*>(a.x) + tok * a.xs;
  T* o = static_cast<T*>(a.out) + tok * a.os;
  constexpr int W = INTER && V == 1 ? 2 : V;  // columns of an item at one place
  const int rot_items = INTER ? 2 * a.half / W : a.half / W;
  const int items = rot_items + (a.copy ? (a.d_h - 2 * a.half) / V : 0);
  for (int u = threadIdx.x; u < a.heads * items; u += blockDim.x) {
    const int h = u / items, i = u - h * items;
    const long long base = (long long)h * a.d_h;
    if (i >= rot_items) {  // past the rotated part
      const long long c = base + 2 * a.half + (long long)(i - rot_items) * V;
      float v[V];
      load_vals<T, V>(x + c, v);
      store_vals<T, V>(o + c, v);
    } else if constexpr (INTER) {
      const long long c = base + (long long)i * W;
      float v[W], y[W];
      if constexpr (V == 1) {
        v[0] = to_f32(x[c]);
        v[1] = to_f32(x[c + 1]);
      } else {
        load_vals<T, V>(x + c, v);
      }
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        const float2 cs = tab[i * (W / 2) + j];
        rope_pair(v[2 * j], v[2 * j + 1], cs, y[2 * j], y[2 * j + 1]);
      }
      if constexpr (V == 1) {
        from_f32(y[0], o[c]);
        from_f32(y[1], o[c + 1]);
      } else {
        store_vals<T, V>(o + c, y);
      }
    } else {
      const long long c0 = base + (long long)i * V, c1 = c0 + a.half;
      float v0[V], v1[V], y0[V], y1[V];
      load_vals<T, V>(x + c0, v0);
      load_vals<T, V>(x + c1, v1);
#pragma unroll
      for (int j = 0; j < V; ++j) rope_pair(v0[j], v1[j], tab[i * V + j], y0[j], y1[j]);
      store_vals<T, V>(o + c0, y0);
      store_vals<T, V>(o + c1, y1);
    }
  }
}

template <typename T>
cudaError_t launch_rope(const RopeArgs& a, int B, bool inter, bool vec, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  void (*fn)(RopeArgs) = inter ? (vec ? rope_kernel<T, V, true> : rope_kernel<T, 1, true>)
                               : (vec ? rope_kernel<T, V, false> : rope_kernel<T, 1, false>);
  return launch_pdl(fn, dim3((unsigned)((long long)B * a.T)), dim3(256), 0, s, a);
}

}  // namespace
}  // namespace dlite

extern "C" int dlite_rope_table(const dlite_rope_config* c, int n_pos, float* table, dlite_stream_t stream) {
  if (!c || !table || ((uintptr_t)table & 7) || n_pos < 1) return DLITE_ERR_INVALID_ARG;
  if (c->rot < 2 || c->rot > 256 || c->rot % 2) return DLITE_ERR_UNSUPPORTED_SHAPE;
  if (!(c->theta > 1.0) || isinf(c->theta) || !(c->attn_factor >= 0.0) || isinf(c->attn_factor)) return DLITE_ERR_INVALID_ARG;
  if (c->scaling < DLITE_ROPE_PLAIN || c->scaling > DLITE_ROPE_YARN) return DLITE_ERR_INVALID_ARG;
  if (c->scaling != DLITE_ROPE_PLAIN && (!(c->factor >= 1.0) || isinf(c->factor))) return DLITE_ERR_INVALID_ARG;
  if (c->scaling == DLITE_ROPE_NTK && c->rot < 4) return DLITE_ERR_UNSUPPORTED_SHAPE;
  if (c->scaling == DLITE_ROPE_YARN &&
      (!(c->orig_len > 0.0) || isinf(c->orig_len) || !(c->beta_slow > 0.0) || !(c->beta_fast > c->beta_slow) ||
       isinf(c->beta_fast)))
    return DLITE_ERR_INVALID_ARG;
  const int half = c->rot / 2;
  const double rot = c->rot;
  double theta = c->theta, m = 1.0, lo = 0.0, hi = 0.0;
  if (c->scaling == DLITE_ROPE_NTK) theta *= pow(c->factor, rot / (rot - 2.0));
  if (c->scaling == DLITE_ROPE_YARN) {
    const double k = rot / (2.0 * log(c->theta)), two_pi = 6.283185307179586;
    lo = std::max(floor(k * log(c->orig_len / (two_pi * c->beta_fast))), 0.0);
    hi = std::min(ceil(k * log(c->orig_len / (two_pi * c->beta_slow))), rot - 1.0);
    m = 0.1 * log(c->factor) + 1.0;
  }
  if (c->attn_factor > 0.0) m = c->attn_factor;
  dlite::RopeFreq fr = {};
  for (int i = 0; i < half; ++i) {
    double f = pow(theta, -2.0 * i / rot);
    if (c->scaling == DLITE_ROPE_LINEAR) f /= c->factor;
    if (c->scaling == DLITE_ROPE_YARN) {
      // a ramp of no width (lo >= hi) is a step at lo
      const double r = hi > lo ? std::min(std::max((i - lo) / (hi - lo), 0.0), 1.0) : (i > lo ? 1.0 : 0.0);
      f = f * (1.0 - r) + f / c->factor * r;
    }
    fr.f[i] = f;
  }
  const long long n = (long long)n_pos * half;
  const unsigned grid = (unsigned)std::min<long long>((n + 255) / 256, 16LL * dlite::device_sms());
  return dlite::launch_status(dlite::launch_pdl(dlite::rope_table_kernel, dim3(grid), dim3(256), 0, (cudaStream_t)stream, fr,
                                                half, n_pos, m, reinterpret_cast<float2*>(table)));
}

extern "C" int dlite_rope(const dlite_rope_args* g, dlite_stream_t stream) {
  if (!g || !g->x || !g->out || !g->pos || !g->table) return DLITE_ERR_INVALID_ARG;
  if (g->B < 1 || g->T < 1 || g->heads < 1 || g->n_pos < 1) return DLITE_ERR_INVALID_ARG;
  if (g->dtype != DLITE_F32 && g->dtype != DLITE_BF16) return DLITE_ERR_INVALID_ARG;
  if (g->layout != DLITE_ROPE_HALF && g->layout != DLITE_ROPE_INTERLEAVED) return DLITE_ERR_INVALID_ARG;
  if (g->d_h < 2 || g->d_h > 1024 || g->rot < 2 || g->rot % 2 || g->rot > g->d_h || g->rot > 256 || g->heads > 65536 ||
      (long long)g->B * g->T > 0x7fffffffLL)
    return DLITE_ERR_UNSUPPORTED_SHAPE;
  const long long cols = (long long)g->heads * g->d_h;
  if (g->x_stride < cols || g->out_stride < cols) return DLITE_ERR_INVALID_ARG;
  if (g->out == g->x && g->out_stride != g->x_stride) return DLITE_ERR_INVALID_ARG;
  const int es = g->dtype == DLITE_F32 ? 4 : 2, V = 16 / es;
  if (((uintptr_t)g->x | (uintptr_t)g->out) % es || (uintptr_t)g->pos % 8 || (uintptr_t)g->table % 8 ||
      !dlite::aligned4(g->n_rows, g->status))
    return DLITE_ERR_INVALID_ARG;
  const bool inter = g->layout == DLITE_ROPE_INTERLEAVED;
  // 16-byte accesses need every item to start on 16 bytes: rows, heads, the rotated part and (half layout) its half
  const bool vec = !(((uintptr_t)g->x | (uintptr_t)g->out) & 15) && g->x_stride % V == 0 && g->out_stride % V == 0 &&
                   g->d_h % V == 0 && g->rot % (inter ? V : 2 * V) == 0;
  dlite::RopeArgs a = {};
  a.T = g->T;
  a.heads = g->heads;
  a.d_h = g->d_h;
  a.half = g->rot / 2;
  a.n_pos = g->n_pos;
  a.copy = g->out != g->x;
  a.x = g->x;
  a.xs = g->x_stride;
  a.out = g->out;
  a.os = g->out_stride;
  a.pos = g->pos;
  a.n_rows = g->n_rows;
  a.table = reinterpret_cast<const float2*>(g->table);
  a.status = g->status;
  const cudaStream_t s = (cudaStream_t)stream;
  return dlite::launch_status(g->dtype == DLITE_F32 ? dlite::launch_rope<float>(a, g->B, inter, vec, s)
                                                    : dlite::launch_rope<dlite::bf16>(a, g->B, inter, vec, s));
}
