// Append to and read from the paged 4-bit cache of the target side.
//
// Append: one CTA per (page a request's new rows touch, KV head, keys or values, request). An
// item is two blocks of 16 columns: of a key, a block and the block of its rotation
// partners, so that a column is loaded and a table entry read once; of the values, a
// block of two neighbouring tokens, whose codes share bytes. Keys go straight out (8 bytes
// of a token's row). Value codes are transposed through shared memory: a page that is filled whole
// leaves as 16-byte stores, else each byte is one thread's, and a byte whose
// other token is old is read and merged. Bound: for prompts a CTA's loads, which nothing covers since it loads,
// computes and stores once (53% of the issue slots, 42% of the warps active, loads the first stall): 8,192 bf16 tokens of 8 heads of 128,
// rotated, 22 us, 2.1 TB/s (35 us with a division per value and a block per thread); launch latency and two
// dependent loads (position, page id) for a token (2.8 us).
//
// Read: the CTA fetches its record with one bulk copy (9 KB at d_h 128) and decodes the
// rows asked for out of shared memory; two tokens' values share bytes and are decoded together (the 8,192 tokens: 12 us,
// 3.5 TB/s, a byte at a time out of shared memory; one 2.2 us).
#include <algorithm>

#include "kv_page.cuh"
#include "rope.cuh"
#include "tc_device.cuh"

namespace dlite {
namespace {

struct AppendArgs {
  uint8_t* pages;
  const int32_t* bt;
  int n_pages, n_kv, max_pages;
  int T, half, inter, n_pos;
  float k_inv, v_inv;  // 2^-exp
  const void *k, *v;
  long long ks, vs;
  const int64_t* pos;
  const int32_t* n_rows;
  const float2* table;  // null: no rotation
  int pairs;            // blocks of 16 columns whose partners fill a block too (16-byte access, halves): 0 or rot / 32
  int* status;
};

// 8 consecutive values as float: 16-byte accesses (VEC) or one by one
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, float* v) {
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(p[i]);
  } else if constexpr (sizeof(T) == 2) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
  } else {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

// Columns c .. c + 7 of a key row after the rotation. VEC: 8 columns lie on one side of
// every border (the halves and the rotated part are multiples of 8 columns).
template <typename T, bool VEC>
__device__ __forceinline__ void rotated8(const T* row, int c, int half, bool inter, const float2* tab, float* y) {
  if constexpr (VEC) {
    load8<T, VEC>(row + c, y);
    if (!tab || c >= 2 * half) return;
    if (inter) {
#pragma unroll
      for (int j = 0; j < 4; ++j) rope_pair(y[2 * j], y[2 * j + 1], tab[c / 2 + j], y[2 * j], y[2 * j + 1]);
    } else {
      const bool first = c < half;
      float o[8];
      load8<T, VEC>(row + (first ? c + half : c - half), o);
      const float2* tb = tab + (first ? c : c - half);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 cs = tb[j];
        float y0, y1;
        rope_pair(first ? y[j] : o[j], first ? o[j] : y[j], cs, y0, y1);
        y[j] = first ? y0 : y1;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int cc = c + j;
      y[j] = to_f32(row[cc]);
      if (!tab || cc >= 2 * half) continue;
      const int i = inter ? cc >> 1 : (cc < half ? cc : cc - half);
      const bool first = inter ? !(cc & 1) : cc < half;
      const float o = to_f32(row[inter ? cc ^ 1 : (first ? cc + half : cc - half)]);
      float y0, y1;
      rope_pair(first ? y[j] : o, first ? o : y[j], tab[i], y0, y1);
      y[j] = first ? y0 : y1;
    }
  }
}

// The rows of request b in page `page` (the request's page_i-th touched one): tokens [lo, hi)
// of the page, from row t0 of the call on. False: none.
struct Span {
  long long page;
  int lo, hi, t0;
};
__device__ __forceinline__ bool page_span(const int64_t* pos, const int32_t* n_rows, int T, int b, int page_i, Span& s) {
  const long long p0 = first_position(pos, b);
  const int n = n_rows ? min(max(n_rows[b], 0), T) : T;
  s.page = (p0 >> 6) + page_i;
  const long long first = max(p0, s.page * 64), last = min(p0 + n, s.page * 64 + 64);
  if (first >= last) return false;
  s.lo = (int)(first - s.page * 64);
  s.hi = (int)(last - s.page * 64);
  s.t0 = (int)(first - p0);
  return true;
}

template <typename T, int DH, bool VEC>
__global__ void __launch_bounds__(256, 4) kv_append_kernel(AppendArgs a) {
  constexpr int NB = DH / 16;
  constexpr int BLK = 16 * 32 + 16;  // bytes of a block of columns; + 16: blocks start in banks of their own
  __shared__ __align__(16) uint8_t vc[NB * BLK];  // the page's value codes, as they go out
  pdl_trigger();
  pdl_wait();
  const int h = blockIdx.y >> 1, b = blockIdx.z, tid = threadIdx.x, nthr = blockDim.x;
  Span sp;
  if (!page_span(a.pos, a.n_rows, a.T, b, blockIdx.x, sp)) return;
  int id = -1;
  if (sp.page >= 0 && sp.page < a.max_pages) id = a.bt[(size_t)b * a.max_pages + sp.page];
  if (id < 0 || id >= a.n_pages) {
    if (tid == 0) flag_status(a.status, kDevBounds);
    return;
  }
  uint8_t* rec = a.pages + ((size_t)id * a.n_kv + h) * kv::rec_bytes(DH);
  const int nt = sp.hi - sp.lo, b0 = sp.lo >> 1, nb = ((sp.hi + 1) >> 1) - b0;  // tokens; bytes (pairs of tokens) of a column
  bool bad = false;
  float v[2][16];
  uint2 codes[2];
  uint32_t scale[2];
  if (blockIdx.y & 1) {  // a token's key, two blocks of 16 columns
    for (int u = tid; u < nt * (NB / 2); u += nthr) {
      const int i = u / (NB / 2), q = u % (NB / 2), tok = sp.lo + i;
      const bool pair = q < a.pairs;  // the blocks are each other's partners
      const int j0 = pair ? q : 2 * q, j1 = pair ? q + a.pairs : 2 * q + 1;
      const T* row = static_cast<const T*>(a.k) + ((long long)b * a.T + sp.t0 + i) * a.ks + (long long)h * DH;
      const float2* tab = nullptr;
      if (a.table) {
        long long p = sp.page * 64 + tok;
        if (p >= a.n_pos) {
          p = a.n_pos - 1;
          flag_status(a.status, kDevBounds);
        }
        tab = a.table + p * a.half;
      }
      if (VEC && pair) {
        load8<T, VEC>(row + 16 * j0, v[0]);
        load8<T, VEC>(row + 16 * j0 + 8, v[0] + 8);
        load8<T, VEC>(row + 16 * j1, v[1]);
        load8<T, VEC>(row + 16 * j1 + 8, v[1] + 8);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float4 cs = *reinterpret_cast<const float4*>(tab + 16 * j0 + e);
          rope_pair(v[0][e], v[1][e], make_float2(cs.x, cs.y), v[0][e], v[1][e]);
          rope_pair(v[0][e + 1], v[1][e + 1], make_float2(cs.z, cs.w), v[0][e + 1], v[1][e + 1]);
        }
      } else {
        rotated8<T, VEC>(row, 16 * j0, a.half, a.inter, tab, v[0]);
        rotated8<T, VEC>(row, 16 * j0 + 8, a.half, a.inter, tab, v[0] + 8);
        rotated8<T, VEC>(row, 16 * j1, a.half, a.inter, tab, v[1]);
        rotated8<T, VEC>(row, 16 * j1 + 8, a.half, a.inter, tab, v[1] + 8);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j = x ? j1 : j0;
        bad |= kv::quantise16(v[x], a.k_inv, codes[x], scale[x]);
        *reinterpret_cast<uint2*>(rec + tok * (DH / 2) + 8 * j) = codes[x];
        rec[kv::ks_off(DH) + tok * NB + j] = (uint8_t)scale[x];
      }
    }
    if (bad) flag_status(a.status, kDevNonfinite);
    return;
  }
  for (int u = tid; u < nb * NB; u += nthr) {  // a block of 16 value columns, two tokens
    const int j = u % NB, by = b0 + u / NB;
    const int i0 = 2 * by - sp.lo;  // -1: the even token is not new
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (i0 + x >= 0 && i0 + x < nt) {
        const T* row = static_cast<const T*>(a.v) + ((long long)b * a.T + sp.t0 + i0 + x) * a.vs + (long long)h * DH + 16 * j;
        load8<T, VEC>(row, v[x]);
        load8<T, VEC>(row + 8, v[x] + 8);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[x][e] = 0.f;
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      bad |= kv::quantise16(v[x], a.v_inv, codes[x], scale[x]);
      if (i0 + x >= 0 && i0 + x < nt) rec[kv::vs_off(DH) + j * 64 + 2 * by + x] = (uint8_t)scale[x];
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {  // nibbles of 8 columns of both tokens -> a byte a column
      const uint32_t c0 = w ? codes[0].y : codes[0].x, c1 = w ? codes[1].y : codes[1].x;
      const uint32_t even = (c0 & 0x0f0f0f0fu) | ((c1 & 0x0f0f0f0fu) << 4), uneven = ((c0 >> 4) & 0x0f0f0f0fu) | (c1 & 0xf0f0f0f0u);
#pragma unroll
      for (int e = 0; e < 8; ++e) vc[j * BLK + (8 * w + e) * 32 + by] = (uint8_t)((e & 1 ? uneven : even) >> (4 * (e & ~1)));
    }
  }
  if (bad) flag_status(a.status, kDevNonfinite);
  __syncthreads();
  uint8_t* vd = rec + kv::v_off(DH);
  if (nt == 64) {
    for (int u = tid; u < DH * 2; u += nthr)
      reinterpret_cast<uint4*>(vd)[u] = *reinterpret_cast<const uint4*>(vc + (u >> 5) * BLK + (u & 31) * 16);
  } else {
    for (int u = tid; u < DH * nb; u += nthr) {
      const int d = u / nb, by = b0 + (u - d * nb), at = d * 32 + by;
      const uint8_t code = vc[(d >> 4) * BLK + (d & 15) * 32 + by];
      // the byte's old token, if it has one, stays
      const uint32_t old = 2 * by < sp.lo ? 0x0fu : 2 * by + 1 >= sp.hi ? 0xf0u : 0u;
      vd[at] = (uint8_t)(old ? (vd[at] & old) | (code & ~old) : code);
    }
  }
}

struct ReadArgs {
  const uint8_t* pages;
  const int32_t* bt;
  int n_pages, n_kv, max_pages, T;
  float k_scale, v_scale;  // 2^exp
  void *k, *v;
  long long ks, vs;
  const int64_t* pos;
  const int32_t* n_rows;
  int* status;
};

__device__ __forceinline__ void put(float x, float& y) { y = x; }
__device__ __forceinline__ void put(float x, bf16& y) { y = __float2bfloat16_rn(x); }

// 16 decoded values to p: 16-byte stores where p allows them
template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&v)[16], bool vec) {
  T o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) put(v[i], o[i]);
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(o)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = o[i];
  }
}

// The values of 8 codes (nibble e of w)
__device__ __forceinline__ void decode8(uint32_t w, float s, float* v) {
  const uint32_t p[4] = {kv::fp4x2_of<0>(w), kv::fp4x2_of<1>(w), kv::fp4x2_of<2>(w), kv::fp4x2_of<3>(w)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
}

template <typename T, int DH>
__global__ void __launch_bounds__(256) kv_read_kernel(ReadArgs a, bool vec) {
  constexpr int NB = DH / 16;
  __shared__ __align__(128) uint8_t rec[kv::rec_bytes(DH)];
  __shared__ __align__(8) uint64_t bar;
  pdl_trigger();
  pdl_wait();
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, nthr = blockDim.x;
  Span sp;
  if (!page_span(a.pos, a.n_rows, a.T, b, blockIdx.x, sp)) return;
  int id = -1;
  if (sp.page >= 0 && sp.page < a.max_pages) id = a.bt[(size_t)b * a.max_pages + sp.page];
  if (id < 0 || id >= a.n_pages) {
    if (tid == 0) flag_status(a.status, kDevBounds);
    return;
  }
  const uint32_t bs = tc::su32(&bar);
  if (tid == 0) {
    tc::mbar_init(bs, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tc::mbar_expect_tx(bs, kv::rec_bytes(DH));
    tc::bulk_load(tc::su32(rec), a.pages + ((size_t)id * a.n_kv + h) * kv::rec_bytes(DH), kv::rec_bytes(DH), bs);
  }
  __syncthreads();
  if (!__syncthreads_and(tc::mbar_wait(bs, 0, a.status))) {  // the copy never landed: give it one more bounded wait, leave
    if (tid == 0) tc::mbar_wait(bs, 0, a.status);
    __syncthreads();
    return;
  }
  const int nt = sp.hi - sp.lo, b0 = sp.lo >> 1, nb = ((sp.hi + 1) >> 1) - b0;  // tokens; bytes (pairs of tokens) of a column
  const long long row0 = (long long)b * a.T + sp.t0 - sp.lo, c0 = (long long)h * DH;
  const int k_items = nt * NB;
  for (int u = tid; u < k_items + nb * NB; u += nthr) {
    float v[16];
    if (u < k_items) {  // 16 key columns of a token
      const int tok = sp.lo + u / NB, j = u % NB;
      const uint2 w = *reinterpret_cast<const uint2*>(rec + tok * (DH / 2) + 8 * j);
      const float s = kv::fp8_to_f32(rec[kv::ks_off(DH) + tok * NB + j]) * a.k_scale;
      decode8(w.x, s, v);
      decode8(w.y, s, v + 8);
      store16(static_cast<T*>(a.k) + (row0 + tok) * a.ks + c0 + 16 * j, v, vec);
    } else {  // 16 value columns of two tokens, which share bytes: the pairs of a block side by side
      const int j = (u - k_items) / nb, by = b0 + (u - k_items) - j * nb;
      uint32_t w[2][2] = {{0u, 0u}, {0u, 0u}};  // [token][8 columns]
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t x = rec[kv::v_off(DH) + (16 * j + e) * 32 + by];
        w[0][e >> 3] |= (x & 15u) << (4 * (e & 7));
        w[1][e >> 3] |= (x >> 4) << (4 * (e & 7));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = 2 * by + i;
        if (tok < sp.lo || tok >= sp.hi) continue;
        const float s = kv::fp8_to_f32(rec[kv::vs_off(DH) + j * 64 + tok]) * a.v_scale;
        decode8(w[i][0], s, v);
        decode8(w[i][1], s, v + 8);
        store16(static_cast<T*>(a.v) + (row0 + tok) * a.vs + c0 + 16 * j, v, vec);
      }
    }
  }
}

// CTAs along the pages: as many as T rows can touch from any first position
inline unsigned touched_pages(int T) { return (unsigned)((T + 2 * kv::kPage - 2) / kv::kPage); }
// Threads: 256 once a page holds more items than 128 threads take in a turn
inline unsigned cta_threads(int T, int d_h) { return std::min(T, kv::kPage) * (d_h / 16) * 2 > 128 ? 256 : 128; }

}  // namespace
}  // namespace dlite

extern "C" int dlite_kv_append(const dlite_kv_append_args* g, dlite_stream_t stream) {
  using namespace dlite;
  if (!g || !g->k || !g->v) return DLITE_ERR_INVALID_ARG;
  const dlite_kv_cache& c = g->cache;
  if (const int rc = kv::check_cache(c, g->B, g->T, g->pos, g->n_rows, g->status)) return rc;
  if (g->dtype != DLITE_F32 && g->dtype != DLITE_BF16) return DLITE_ERR_INVALID_ARG;
  const int es = g->dtype == DLITE_F32 ? 4 : 2;
  const long long cols = (long long)c.n_kv * c.d_h;
  if (g->k_stride < cols || g->v_stride < cols || ((uintptr_t)g->k | (uintptr_t)g->v) % es) return DLITE_ERR_INVALID_ARG;
  if (g->table) {
    if ((g->layout != DLITE_ROPE_HALF && g->layout != DLITE_ROPE_INTERLEAVED) || g->n_pos < 1 || (uintptr_t)g->table % 8)
      return DLITE_ERR_INVALID_ARG;
    if (g->rot < 2 || g->rot % 2 || g->rot > c.d_h) return DLITE_ERR_UNSUPPORTED_SHAPE;
  }
  AppendArgs a = {};
  a.pages = static_cast<uint8_t*>(c.pages);
  a.bt = c.block_table;
  a.n_pages = c.n_pages;
  a.n_kv = c.n_kv;
  a.max_pages = c.max_pages;
  a.T = g->T;
  a.half = g->table ? g->rot / 2 : 0;
  a.inter = g->layout == DLITE_ROPE_INTERLEAVED;
  a.n_pos = g->n_pos;
  a.k_inv = ldexpf(1.f, -c.k_exp);
  a.v_inv = ldexpf(1.f, -c.v_exp);
  a.k = g->k;
  a.ks = g->k_stride;
  a.v = g->v;
  a.vs = g->v_stride;
  a.pos = g->pos;
  a.n_rows = g->n_rows;
  a.table = reinterpret_cast<const float2*>(g->table);
  a.status = g->status;
  // 16-byte loads: rows on 16 bytes, and (rotated keys) borders at multiples of 8 columns
  const int V = 16 / es;
  const bool vec = !(((uintptr_t)g->k | (uintptr_t)g->v) & 15) && g->k_stride % V == 0 && g->v_stride % V == 0 &&
                   (!g->table || g->rot % (a.inter ? 8 : 16) == 0);
  a.pairs = vec && g->table && !a.inter && g->rot % 32 == 0 && (uintptr_t)g->table % 16 == 0 ? g->rot / 32 : 0;
  void (*fn)(AppendArgs);
  if (g->dtype == DLITE_F32)
    fn = c.d_h == 128 ? (vec ? kv_append_kernel<float, 128, true> : kv_append_kernel<float, 128, false>)
                      : (vec ? kv_append_kernel<float, 64, true> : kv_append_kernel<float, 64, false>);
  else
    fn = c.d_h == 128 ? (vec ? kv_append_kernel<bf16, 128, true> : kv_append_kernel<bf16, 128, false>)
                      : (vec ? kv_append_kernel<bf16, 64, true> : kv_append_kernel<bf16, 64, false>);
  return launch_status(launch_pdl(fn, dim3(touched_pages(g->T), 2 * c.n_kv, g->B), dim3(cta_threads(g->T, c.d_h)), 0,
                                  (cudaStream_t)stream, a));
}

extern "C" int dlite_kv_read(const dlite_kv_read_args* g, dlite_stream_t stream) {
  using namespace dlite;
  if (!g || !g->k_out || !g->v_out) return DLITE_ERR_INVALID_ARG;
  const dlite_kv_cache& c = g->cache;
  if (const int rc = kv::check_cache(c, g->B, g->T, g->pos, g->n_rows, g->status)) return rc;
  if (g->dtype != DLITE_F32 && g->dtype != DLITE_BF16) return DLITE_ERR_INVALID_ARG;
  const int es = g->dtype == DLITE_F32 ? 4 : 2, V = 16 / es;
  const long long cols = (long long)c.n_kv * c.d_h;
  if (g->k_stride < cols || g->v_stride < cols || ((uintptr_t)g->k_out | (uintptr_t)g->v_out) % es) return DLITE_ERR_INVALID_ARG;
  ReadArgs a = {};
  a.pages = static_cast<const uint8_t*>(c.pages);
  a.bt = c.block_table;
  a.n_pages = c.n_pages;
  a.n_kv = c.n_kv;
  a.max_pages = c.max_pages;
  a.T = g->T;
  a.k_scale = ldexpf(1.f, c.k_exp);
  a.v_scale = ldexpf(1.f, c.v_exp);
  a.k = g->k_out;
  a.ks = g->k_stride;
  a.v = g->v_out;
  a.vs = g->v_stride;
  a.pos = g->pos;
  a.n_rows = g->n_rows;
  a.status = g->status;
  const bool vec = !(((uintptr_t)g->k_out | (uintptr_t)g->v_out) & 15) && g->k_stride % V == 0 && g->v_stride % V == 0;
  void (*fn)(ReadArgs, bool) = g->dtype == DLITE_F32 ? (c.d_h == 128 ? kv_read_kernel<float, 128> : kv_read_kernel<float, 64>)
                                                     : (c.d_h == 128 ? kv_read_kernel<bf16, 128> : kv_read_kernel<bf16, 64>);
  return launch_status(launch_pdl(fn, dim3(touched_pages(g->T), c.n_kv, g->B), dim3(cta_threads(g->T, c.d_h)), 0,
                                  (cudaStream_t)stream, a, vec));
}
