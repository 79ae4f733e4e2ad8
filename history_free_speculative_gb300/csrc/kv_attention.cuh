// Shared parts of the paged-cache attention kernels: how the work is cut, and
// how the pieces of a tile are written and joined.
//
// A segment is one tile of query rows of one (request, KV head); its pages are counted in units (UP pages). Stream form:
// the units of all segments, in order, are cut into equal runs of `quota` units, one per CTA, whatever the lengths of
// the requests; a CTA walks the pieces of segments in its run. Every
// segment begins with `change` units without pages, which stand for the time that a change of pieces takes. A piece that is its whole
// segment writes the output; other pieces leave (max, sum, unnormalised output) in the workspace, at most two a CTA, and the
// join kernel adds them up in order. Every CTA works the cut out for itself from pos and n_rows, so that lengths stay on the device.
// Whole form (segments that are short by the table's width, or too many for the list of prefix sums): CTAs take whole
// segments in turn.
#pragma once

#include "kv_page.cuh"
#include "tc_device.cuh"

namespace dlite {
namespace kv {

constexpr int kMaxList = 2048;  // row tiles of all requests in the stream form

// Weights are kept as 2^((s - ref) factor + exp): s a raw score (the products' sum), ref the row's reference, a raw score too, factor what
// takes raw scores to powers of two. The difference comes before the factor: with the reference as a power of two, its rounding
// (half a step of the score) moved the largest weight itself, and scores of 2^26 and more passed f16's range.
constexpr float kWeightExp = 14.f, kTcWeightExp = 6.f;

struct AttnArgs {
  const uint8_t* pages;
  const int32_t* bt;
  int n_pages, n_kv, max_pages;
  int B, T, n_q, group, window;
  int row_tiles;        // of a KV head's group x T rows
  int unit;             // pages of a unit
  int min_quota;        // units a CTA takes at least (stream form)
  int change;           // what a change of pieces costs a CTA, in units
  int stream;           // 1: stream form
  float scale_mant;     // scale log2(e) 2^k_exp = scale_mant 2^scale_exp, scale_mant in [1/2, 1)
  int scale_exp;
  float v_scale;        // 2^v_exp
  float weight_exp;     // weights are kept as 2^(s - m + weight_exp)
  const void* q;
  long long qs;
  void* out;
  long long os;
  float* lse;
  const int64_t* pos;
  const int32_t* n_rows;
  float* part_o;    // [CTA][2][row][d_h]: slot 0 a piece that began before the CTA's run, 1 one that goes on after it
  float2* part_ml;  // [CTA][2][row]: running maximum (log2 units) and sum
  int2* joins;      // [CTA]: segment that begins in the CTA's run and goes on after it, and its number of pieces (0: none)
  int vec;          // q and out rows on 16 bytes
  int* status;
};

// How a query row becomes f16: multiplied by f0 f1 = 2^e2, which takes its largest element into [2^14, 2^15) (two factors, since e2 goes from -113
// to 163), and factor, which takes the row's raw scores to powers of two. The factor's exponent is worked out before its value: scale, k_exp
// and e2 may each pass float32's range where their sum does not. Below 2^-126 all weights are 1 to float32's precision; it
// stays above 0 so that a masked -inf stays -inf. Above 2^127 all but scores near 0 are past float32.
struct RowScale {
  float f0, f1, factor;
};
__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }  // -126 <= k <= 127
__device__ __forceinline__ RowScale row_scale(const AttnArgs& a, float amax) {  // amax finite
  const int e2 = amax > 0.f ? 14 - ilogbf(amax) : 0, h = e2 >> 1;
  return {pow2(h), pow2(e2 - h), a.scale_mant * pow2(min(max(a.scale_exp - e2, -125), 127))};
}

// One tile of rows of a request: rows [r0, r1) (row r is token r / group, head r % group), keys [key_beg, key_end) that some
// row may see, the pages they lie in.
struct Tile {
  long long p0, cap;
  int r0, r1, t_lo, t_hi, key_beg, key_end, pg0, np;
};
template <int R>
__device__ __forceinline__ Tile tile_of(const AttnArgs& a, int b, int rt) {
  Tile t;
  const int n = a.n_rows ? min(max(a.n_rows[b], 0), a.T) : a.T;
  t.p0 = first_position(a.pos, b);
  t.cap = (long long)a.max_pages * kPage;
  t.r0 = rt * R;
  t.r1 = min(t.r0 + R, n * a.group);
  t.t_lo = t.r0 / a.group;
  t.t_hi = (t.r1 - 1) / a.group;
  t.key_end = (int)min(max(t.p0 + t.t_hi + 1, 0LL), t.cap);
  t.key_beg = a.window ? (int)min(max(t.p0 + t.t_lo - a.window + 1, 0LL), t.cap) : 0;
  t.pg0 = t.key_beg / kPage;
  t.np = t.key_end > t.key_beg ? (t.key_end + kPage - 1) / kPage - t.pg0 : 0;
  return t;
}
// Units of a tile: one at least if it has rows (a row without keys is written too)
__device__ __forceinline__ int units_of(const Tile& t, int unit) {
  return t.r0 < t.r1 ? max(1, (t.np + unit - 1) / unit) : 0;
}

struct Piece {
  int j, h;        // row tile of all requests (b row_tiles + rt), KV head
  int u0, u1, nu;  // units [u0, u1) of the segment's nu
  __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == nu; }
};

// prefix [row tiles + 1]: units of the row tiles before (of one KV head), with those of the changes. All threads of the CTA; ends with a barrier.
template <int R>
__device__ __forceinline__ void build_prefix(const AttnArgs& a, int* prefix) {
  const int J = a.B * a.row_tiles;
  for (int j = threadIdx.x; j < J; j += blockDim.x) {
    const int units = units_of(tile_of<R>(a, j / a.row_tiles, j % a.row_tiles), a.unit);
    prefix[j + 1] = units ? units + a.change : 0;
  }
  if (threadIdx.x == 0) prefix[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    int carry = 0;
    for (int j0 = 0; j0 < J; j0 += 32) {
      const int j = j0 + threadIdx.x;
      int v = j < J ? prefix[j + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, v, o);
        if ((int)threadIdx.x >= o) v += w;
      }
      v += carry;
      if (j < J) prefix[j + 1] = v;
      carry = __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
}

// Walks the pieces of this CTA.
template <int R>
struct Pieces {
  const AttnArgs& a;
  const int* prefix;
  int J;
  uint32_t u, end, quota;  // the host takes the stream form where all units are below 2^31
  int j;
  __device__ __forceinline__ Pieces(const AttnArgs& args, const int* pre) : a(args), prefix(pre) {
    J = a.B * a.row_tiles;
    j = 0;
    if (a.stream) {
      const uint32_t U = (uint32_t)prefix[J] * a.n_kv;
      quota = max((U + gridDim.x - 1) / gridDim.x, (uint32_t)a.min_quota);
      u = min(quota * blockIdx.x, U);
      end = min(u + quota, U);
      int lo = 0, hi = J;  // last j with prefix[j] n_kv <= u
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((uint32_t)prefix[mid] * a.n_kv <= u)
          lo = mid;
        else
          hi = mid;
      }
      j = lo;
    } else {
      u = blockIdx.x;
      end = (uint32_t)J * a.n_kv;
    }
  }
  __device__ __forceinline__ bool next(Piece& p) {
    if (a.stream) {
      while (u < end) {
        while ((uint32_t)prefix[j + 1] * a.n_kv <= u) ++j;
        const uint32_t rem = u - (uint32_t)prefix[j] * a.n_kv, all = prefix[j + 1] - prefix[j];
        const int h = (int)(rem / all);
        const int v0 = (int)(rem - h * all), v1 = (int)min(all, v0 + (end - u));
        u += v1 - v0;
        if (v1 <= a.change) continue;  // the run ends before the segment's first page; p stays the last piece
        p.j = j;
        p.h = h;
        p.nu = (int)all - a.change;
        p.u0 = max(v0 - a.change, 0);
        p.u1 = v1 - a.change;
        return true;
      }
      return false;
    }
    for (; u < end; u += gridDim.x) {
      p.j = (int)(u / a.n_kv);
      p.h = (int)(u % a.n_kv);
      p.nu = units_of(tile_of<R>(a, p.j / a.row_tiles, p.j % a.row_tiles), a.unit);
      p.u0 = 0;
      p.u1 = p.nu;
      if (p.nu) {
        u += gridDim.x;
        return true;
      }
    }
    return false;
  }
  // What the join kernel has to know of this CTA: p is its last piece (if any).
  __device__ __forceinline__ int2 join_of(bool any, const Piece& p) const {
    if (!any || p.u0 || p.whole()) return make_int2(0, 0);
    const uint32_t last = (uint32_t)prefix[p.j] * a.n_kv + (uint32_t)(p.h + 1) * (p.nu + a.change) - 1;
    return make_int2(p.j * a.n_kv + p.h, (int)(last / quota) - (int)blockIdx.x + 1);
  }
};
// The pieces of a CTA as a list in shared memory, a batch at a time: one thread walks, one thread a piece works out its
// tile. (Walked by every role of a kernel itself, the divisions and loads were there five times over and sat in every change of pieces.)
struct PieceTile {
  Piece p;
  Tile t;
  int b, rt;
};
constexpr int kBatch = 32;
// Row of the workspace of this CTA's piece p (not its whole segment)
__device__ __forceinline__ size_t part_row(const Piece& p, int R) { return ((size_t)blockIdx.x * 2 + (p.u0 == 0)) * R; }

__device__ __forceinline__ float lse_of(float M, float L, float weight_exp) {
  return L == 0.f ? -INFINITY : (M + (log2f(L) - weight_exp)) * 0.6931471805599453f;
}

// Host side
struct AttnPlan {
  int rows = 16;    // of a tile
  bool tc = false;  // the tcgen05 kernel
  int row_tiles = 1, unit = 1, min_quota = 8, change = 0, grid = 1;
  bool stream = false;
  size_t bytes(int d_h) const { return stream ? (size_t)grid * (2 * rows * ((size_t)d_h * 4 + 8) + 8) : 0; }
};
cudaError_t launch_attention_tc(const AttnArgs& a, const AttnPlan& p, cudaStream_t s);

}  // namespace kv
}  // namespace dlite
