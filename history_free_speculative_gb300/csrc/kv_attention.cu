// Attention of a verification block (or a decoded token) over the paged 4-bit cache.
//
// The query rows of one KV head, (n_q / n_kv) heads x T tokens in token order, are cut into
// tiles of 16 MT rows; how tiles and pages go to CTAs is in kv_attention.cuh. This file has the kernel for
// float32 queries and for heads of 64; bf16 queries with heads of 128 take the tcgen05 kernel (kv_attention_tc.cu).
// A page's record (9 KB at d_h 128) comes with one bulk copy into a ring of shared-memory
// slots; a warp takes every NW-th page of a piece whole, with its own slots, running maximum, sum and output
// (16 MT x d_h fp32 in registers), so warps meet only at a piece's end.
//
// Codes become f16 operands exactly: e2m1 x e4m3 has 6 significant bits between 2^-10 and 2688. Queries are scaled by a power
// of two per row (largest element in [2^14, 2^15)), so a bf16 query is exact in f16 too; a float32 query
// takes two planes (hi + lo, 22 bits). Softmax weights are held as 2^(s - m + 14), in powers of two, so that f16 keeps
// weights down to 2^-38 of the largest; they are rounded to f16 (2^-12 relative, below the bf16 output's 2^-9),
// for float32 outputs as hi + lo. Scores, maxima, sums and outputs are fp32.
// Measured: one float32 token over 500 keys, 4 query and 2 KV heads of 64, 7.0 us with the join; bound by two launches and a
// chain of dependent loads (position, page ids, records). 118,000 keys, 32 query and 8 KV heads, eight tokens: float32 heads of 128 107 us (floor
// 20), float32 heads of 64 62 us, bf16 heads of 64 45 us (floor 10): the products, twice
// as many for float32.
//
// Both products run on mma.sync m16n8k16 straight from the packed bytes: within a product's inner dimension any order
// serves if both operands share it, so each lane takes the codes it can load in one piece.
//   QK^T: lane (g, c) of a warp (g = lane / 4, c = lane % 4) takes columns [c d/4, (c+1) d/4) of key g of an 8-key tile:
//         step i multiplies columns c d/4 + 4i .. + 3. The 8 keys of tile (j, h) of a 32-key half are
//         8 (g / 2) + 4 j + 2 h + g % 2, which puts the scores of keys 8c .. 8c + 7 into lane c: the A operand of
//   PV:   lane (g, c) takes tokens 8c .. 8c + 7 of value column 8 i + g (4 bytes; the cache keeps
//         a column's tokens side by side for this), step j tokens 8c + 4j .. + 3.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "kv_attention.cuh"

namespace dlite {
namespace {

constexpr int kWarps = 8;

using kv::AttnArgs;
using kv::kWeightExp;

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float f16_lo(uint32_t p) { return __half2float(__ushort_as_half((unsigned short)(p & 0xffffu))); }
__device__ __forceinline__ float f16_hi(uint32_t p) { return __half2float(__ushort_as_half((unsigned short)(p >> 16))); }

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <typename T, int DH, int MT>
struct Shape {
  static constexpr int NP = sizeof(T) == 4 ? 2 : 1;  // f16 planes of a query / a weight
  static constexpr int R = 16 * MT;                  // rows of a tile
  static constexpr int REC = kv::rec_bytes(DH);
  static constexpr int SLOTS = (DH == 64 ? 4 : 2) * kWarps;
  static constexpr int STEPS = DH / 16;
  static constexpr int QF = NP * MT * STEPS * 512;   // query fragments, bytes
  static constexpr int LDO = DH + 8;                 // row pitch of the warps' outputs (conflict-free float2 stores)
  static constexpr int SMEM = SLOTS * REC + QF + R * 12 + 2 * kWarps * R * 4 + SLOTS * 12 + (kv::kMaxList + 1) * 4;
  static_assert(kWarps * R * LDO * 4 <= SLOTS * REC, "the warps' outputs share the ring's memory");
  static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
};

// Element i of a query row: bf16 or fp32
template <typename T>
__device__ __forceinline__ void load_q(const T* p, int n, bool vec, float* v) {
  if (vec && sizeof(T) * n == 8) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    const T* e = reinterpret_cast<const T*>(&w);
    for (int i = 0; i < n; ++i) v[i] = to_f32(e[i]);
  } else if (vec && sizeof(T) * n == 16) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const T* e = reinterpret_cast<const T*>(&w);
    for (int i = 0; i < n; ++i) v[i] = to_f32(e[i]);
  } else {
    for (int i = 0; i < n; ++i) v[i] = to_f32(p[i]);
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, const float4& v, bool vec) {
  if constexpr (sizeof(T) == 4) {
    if (vec) {
      *reinterpret_cast<float4*>(p) = v;
      return;
    }
    p[0] = v.x, p[1] = v.y, p[2] = v.z, p[3] = v.w;
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    if (vec) {
      *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
      return;
    }
    p[0] = a.x, p[1] = a.y, p[2] = b.x, p[3] = b.y;
  }
}

// One 32-key half of a page for one warp. key0: first key's position; row_keys: the keys
// [x, y) a row sees, looked at only where MASKED.
template <typename T, int DH, int MT, bool MASKED>
__device__ __forceinline__ void half_page(const uint8_t* rec, int hf, const uint4* qf, const float* row_sc, const int2* row_keys,
                                          int key0, int key_end, float (&m)[MT][2], float (&l)[MT][2],
                                          float (&o)[MT][DH / 8][4]) {
  using S = Shape<T, DH, MT>;
  constexpr int NP = S::NP, STEPS = S::STEPS, KW = DH / 32, NB = DH / 16;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  // keys: codes and scales
  uint32_t kw[4][KW], ks[4][KW / 2];
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) {
    const int key = 32 * hf + 8 * (g >> 1) + 4 * (nt >> 1) + 2 * (nt & 1) + (g & 1);
    const uint8_t* kp = rec + key * (DH / 2) + c * (DH / 8);
    const uint8_t* sp = rec + kv::ks_off(DH) + key * NB + c * (NB / 4);
    if constexpr (DH == 128) {
      const uint4 w = *reinterpret_cast<const uint4*>(kp);
      kw[nt][0] = w.x, kw[nt][1] = w.y, kw[nt][2] = w.z, kw[nt][3] = w.w;
      const uint32_t s2 = kv::fp8x2_to_f16x2(*reinterpret_cast<const uint16_t*>(sp));
      ks[nt][0] = __byte_perm(s2, s2, 0x1010);
      ks[nt][1] = __byte_perm(s2, s2, 0x3232);
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(kp);
      kw[nt][0] = w.x, kw[nt][1] = w.y;
      ks[nt][0] = kv::fp8x2_to_f16x2((uint16_t)(*sp * 0x101u));
    }
  }
  float s[MT][4][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
#pragma unroll
  for (int st = 0; st < STEPS; ++st) {
    uint32_t a[NP][MT][4];
#pragma unroll
    for (int pl = 0; pl < NP; ++pl)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const uint4 w = qf[((pl * MT + mt) * STEPS + st) * 32 + lane];
        a[pl][mt][0] = w.x, a[pl][mt][1] = w.y, a[pl][mt][2] = w.z, a[pl][mt][3] = w.w;
      }
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const uint32_t w = kw[nt][st >> 1], sv = ks[nt][st >> 2];
      const uint32_t b0 = kv::mul_f16x2(st & 1 ? kv::fp4x2_of<2>(w) : kv::fp4x2_of<0>(w), sv);
      const uint32_t b1 = kv::mul_f16x2(st & 1 ? kv::fp4x2_of<3>(w) : kv::fp4x2_of<1>(w), sv);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int pl = 0; pl < NP; ++pl) mma_f16(s[mt][nt], a[pl][mt], b0, b1);
    }
  }
  if constexpr (MASKED) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int2 see = row_keys[mt * 16 + (e >> 1) * 8 + g];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const int key = key0 + 8 * c + 4 * (nt >> 1) + 2 * (nt & 1) + (e & 1);
          if (key < see.x || key >= see.y) s[mt][nt][e] = -INFINITY;
        }
      }
  }
  // online softmax; weights 2^((s - m) sc + 14), m the largest raw score
  uint32_t p[NP][MT][2][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      x0 = fmaxf(x0, fmaxf(s[mt][nt][0], s[mt][nt][1]));
      x1 = fmaxf(x1, fmaxf(s[mt][nt][2], s[mt][nt][3]));
    }
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
    const float sc[2] = {row_sc[mt * 16 + g], row_sc[mt * 16 + 8 + g]};
    const float n0 = fmaxf(m[mt][0], x0), n1 = fmaxf(m[mt][1], x1);
    if (n0 != m[mt][0] || n1 != m[mt][1]) {
      // no key before (m = -inf): nothing to rescale
      const float al0 = n0 == m[mt][0] || m[mt][0] == -INFINITY ? 1.f : tc::ex2_approx((m[mt][0] - n0) * sc[0]);
      const float al1 = n1 == m[mt][1] || m[mt][1] == -INFINITY ? 1.f : tc::ex2_approx((m[mt][1] - n1) * sc[1]);
      l[mt][0] *= al0;
      l[mt][1] *= al1;
#pragma unroll
      for (int dt = 0; dt < DH / 8; ++dt) {
        o[mt][dt][0] *= al0;
        o[mt][dt][1] *= al0;
        o[mt][dt][2] *= al1;
        o[mt][dt][3] *= al1;
      }
      m[mt][0] = n0;
      m[mt][1] = n1;
    }
    // a row with no key yet (m = -inf): every weight is 0
    const float r0 = n0 == -INFINITY ? 0.f : n0, r1 = n1 == -INFINITY ? 0.f : n1;
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = tc::ex2_approx(fmaf(s[mt][nt][e] - (e < 2 ? r0 : r1), sc[e >> 1], kWeightExp));
        if constexpr (MASKED) w[e] = s[mt][nt][e] == -INFINITY ? 0.f : w[e];
      }
      l[mt][0] += w[0] + w[1];
      l[mt][1] += w[2] + w[3];
      const uint32_t h0 = pack_f16(w[0], w[1]), h1 = pack_f16(w[2], w[3]);
      p[0][mt][nt >> 1][(nt & 1) * 2] = h0;
      p[0][mt][nt >> 1][(nt & 1) * 2 + 1] = h1;
      if constexpr (NP == 2) {
        p[1][mt][nt >> 1][(nt & 1) * 2] = pack_f16(w[0] - f16_lo(h0), w[1] - f16_hi(h0));
        p[1][mt][nt >> 1][(nt & 1) * 2 + 1] = pack_f16(w[2] - f16_lo(h1), w[3] - f16_hi(h1));
      }
    }
  }
  // values
  uint32_t sv[4];
#pragma unroll
  for (int dt = 0; dt < DH / 8; ++dt) {
    if (dt % 2 == 0) {
      const uint2 w = *reinterpret_cast<const uint2*>(rec + kv::vs_off(DH) + (dt / 2) * 64 + 32 * hf + 8 * c);
      sv[0] = kv::fp8x2_to_f16x2((uint16_t)w.x);
      sv[1] = kv::fp8x2_to_f16x2((uint16_t)(w.x >> 16));
      sv[2] = kv::fp8x2_to_f16x2((uint16_t)w.y);
      sv[3] = kv::fp8x2_to_f16x2((uint16_t)(w.y >> 16));
      if constexpr (MASKED) {
        // keys past the end hold anything, a NaN scale too: weight 0 times it must stay 0
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int key = key0 + 8 * c + 2 * q;
          sv[q] = key + 1 < key_end ? sv[q] : key < key_end ? sv[q] & 0xffffu : 0u;
        }
      }
    }
    const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + kv::v_off(DH) + (8 * dt + g) * 32 + 16 * hf + 4 * c);
    const uint32_t b0 = kv::mul_f16x2(kv::fp4x2_of<0>(w), sv[0]), b1 = kv::mul_f16x2(kv::fp4x2_of<1>(w), sv[1]);
    const uint32_t b2 = kv::mul_f16x2(kv::fp4x2_of<2>(w), sv[2]), b3 = kv::mul_f16x2(kv::fp4x2_of<3>(w), sv[3]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if constexpr (NP == 2) {
        // The products of a half page apart, the small plane's first, and one rounding add: an MMA cuts its sum off, and over
        // the pages of a warp that added up to a bias of 4 10^-6 (118,000 keys), below a bf16 output's rounding but not a float32's.
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int pl = NP - 1; pl >= 0; --pl) {
          mma_f16(part, p[pl][mt][0], b0, b1);
          mma_f16(part, p[pl][mt][1], b2, b3);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][dt][e] += part[e];
      } else {
        mma_f16(o[mt][dt], p[0][mt][0], b0, b1);
        mma_f16(o[mt][dt], p[0][mt][1], b2, b3);
      }
    }
  }
}

template <typename T, int DH, int MT>
__global__ void __launch_bounds__(32 * kWarps, 1) kv_attention_kernel(const AttnArgs a) {
  using S = Shape<T, DH, MT>;
  constexpr int R = S::R, REC = S::REC, STEPS = S::STEPS, NP = S::NP, LDO = S::LDO, PER = S::SLOTS / kWarps;
  extern __shared__ __align__(128) uint8_t sm[];
  uint8_t* ring = sm;
  uint4* qf = reinterpret_cast<uint4*>(sm + S::SLOTS * REC);
  float* row_sc = reinterpret_cast<float*>(sm + S::SLOTS * REC + S::QF);
  int2* row_keys = reinterpret_cast<int2*>(row_sc + R);
  float* sm_m = reinterpret_cast<float*>(row_keys + R);  // [warp][row]
  float* sm_l = sm_m + kWarps * R;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm_l + kWarps * R);
  int* slot_ok = reinterpret_cast<int*>(full + S::SLOTS);
  int* prefix = slot_ok + S::SLOTS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();  // no early trigger: the grid fills the SMs, and a dependent would only take their slots
  if (a.stream) kv::build_prefix<R>(a, prefix);
  if (tid < S::SLOTS) tc::mbar_init(tc::su32(full + tid), 1);
  if (tid == 0) asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncthreads();

  kv::Pieces<R> walk(a, prefix);
  kv::Piece pc;
  bool any = false, got = true;
  int n_issue = 0, n_take = 0;  // pages this warp has asked for and taken, over all pieces
  while (walk.next(pc)) {
    any = true;
    const int b = pc.j / a.row_tiles, rt = pc.j % a.row_tiles, h = pc.h;
    const kv::Tile t = kv::tile_of<R>(a, b, rt);
    if (tid == 0 && rt == 0 && pc.u0 == 0 && (t.p0 < 0 || t.p0 + (a.n_rows ? min(a.n_rows[b], a.T) : a.T) > t.cap))
      flag_status(a.status, kDevBounds);
    const int pa = t.pg0 + pc.u0, cnt = min(pc.u1, t.np) - pc.u0;
    const int32_t* bt = a.bt + (size_t)b * a.max_pages + pa;
    // lane 0 of a warp: its next page (a hole: an empty slot)
    auto issue = [&](int id) {
      const int slot = warp + kWarps * (n_issue % PER);
      const uint32_t bar = tc::su32(full + slot);
      if (id >= a.n_pages) flag_status(a.status, kDevBounds);
      const bool ok = id >= 0 && id < a.n_pages;
      slot_ok[slot] = ok;
      if (ok) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc::mbar_expect_tx(bar, REC);
        tc::bulk_load(tc::su32(ring + slot * REC), a.pages + ((size_t)id * a.n_kv + h) * REC, REC, bar);
      } else {
        mbar_arrive(bar);
      }
    };
    for (int i = warp; i < cnt && i < PER * kWarps; i += kWarps) {
      if (lane == 0) issue(bt[i]);
      ++n_issue;
    }

    // queries: row r of the tile is token (r0 + r) / group, head (r0 + r) % group of the KV head's
    for (int r = warp; r < R; r += kWarps) {
      constexpr int E = DH / 32;
      float v[E];
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = 0.f;
      if (t.r0 + r < t.r1) {
        const int tk = (t.r0 + r) / a.group, hh = (t.r0 + r) % a.group;
        load_q(static_cast<const T*>(a.q) + ((long long)b * a.T + tk) * a.qs + (long long)(h * a.group + hh) * DH + lane * E, E, a.vec, v);
      }
      float amax = 0.f;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        amax = fmaxf(amax, fabsf(v[i]));
        bad |= !(fabsf(v[i]) <= 3.402823466e38f);
      }
      amax = warp_max(amax);
      bad = __any_sync(0xffffffffu, bad);
      const kv::RowScale rs = kv::row_scale(a, bad ? 0.f : amax);
      if (lane == 0) {
        row_sc[r] = bad ? NAN : rs.factor;
        const long long last = t.p0 + min(t.r0 + r, t.r1 - 1) / a.group;
        row_keys[r] = make_int2(a.window ? (int)min(max(last - a.window + 1, 0LL), t.cap) : 0, (int)min(max(last + 1, 0LL), t.cap));
      }
      const int mt = r / 16, up = (r % 16) >= 8, g = r % 8;
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const int d = lane * E + i, c = d / (DH / 4), st = (d % (DH / 4)) / 4, reg = (d % 4 >= 2 ? 2 : 0) + up;
        const float x0 = bad ? 0.f : v[i] * rs.f0 * rs.f1, x1 = bad ? 0.f : v[i + 1] * rs.f0 * rs.f1;
        const uint32_t hi = pack_f16(x0, x1);
        uint32_t* dst = reinterpret_cast<uint32_t*>(qf + (mt * STEPS + st) * 32 + g * 4 + c) + reg;
        *dst = hi;
        if constexpr (NP == 2) dst[MT * STEPS * 128] = pack_f16(x0 - f16_lo(hi), x1 - f16_hi(hi));
      }
    }
    __syncthreads();

    float m[MT][2], l[MT][2], o[MT][DH / 8][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
      for (int dt = 0; dt < DH / 8; ++dt) o[mt][dt][0] = o[mt][dt][1] = o[mt][dt][2] = o[mt][dt][3] = 0.f;
    }
    // pages wholly inside every row's range need no masks
    const int full_end = (int)min(max(t.p0 + t.t_lo + 1, 0LL), t.cap);
    const int full_beg = a.window ? (int)min(max(t.p0 + t.t_hi - a.window + 1, 0LL), t.cap) : 0;

    for (int i = warp; i < cnt; i += kWarps) {
      const int slot = warp + kWarps * (n_take % PER);
      const bool more = i + PER * kWarps < cnt;
      int id_next = -1;
      if (lane == 0 && more) id_next = bt[i + PER * kWarps];
      // a copy that never lands: no further page is taken, the status says so, the barriers below are kept
      got = got && __all_sync(0xffffffffu, tc::mbar_wait_hint(tc::su32(full + slot), (uint32_t)(n_take / PER) & 1u, a.status));
      ++n_take;
      if (got && slot_ok[slot]) {
        const uint8_t* rec = ring + slot * REC;
        const int key0 = (pa + i) * kv::kPage;
        if (key0 >= full_beg && key0 + kv::kPage <= full_end) {
          half_page<T, DH, MT, false>(rec, 0, qf, row_sc, row_keys, key0, t.key_end, m, l, o);
          half_page<T, DH, MT, false>(rec, 1, qf, row_sc, row_keys, key0 + 32, t.key_end, m, l, o);
        } else {
          half_page<T, DH, MT, true>(rec, 0, qf, row_sc, row_keys, key0, t.key_end, m, l, o);
          if (key0 + 32 < t.key_end) half_page<T, DH, MT, true>(rec, 1, qf, row_sc, row_keys, key0 + 32, t.key_end, m, l, o);
        }
      }
      __syncwarp();
      if (more) {
        if (lane == 0 && got) issue(id_next);
        ++n_issue;
      }
    }

    // the warps' rows joined: maxima, then outputs scaled to the common maximum, summed in warp order
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[mt][e] += __shfl_xor_sync(0xffffffffu, l[mt][e], 1);
        l[mt][e] += __shfl_xor_sync(0xffffffffu, l[mt][e], 2);
        m[mt][e] *= m[mt][e] == -INFINITY ? 1.f : row_sc[mt * 16 + e * 8 + (lane >> 2)];   // a power of two from here on
        if ((lane & 3) == 0) sm_m[warp * R + mt * 16 + e * 8 + (lane >> 2)] = m[mt][e];
      }
    __syncthreads();
    float* ob = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = mt * 16 + e * 8 + (lane >> 2);
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w * R + r]);
        const float f = m[mt][e] == -INFINITY ? 0.f : tc::ex2_approx(m[mt][e] - M);
        if ((lane & 3) == 0) sm_l[warp * R + r] = l[mt][e] * f;
        float* dst = ob + (warp * R + r) * LDO + 2 * (lane & 3);
#pragma unroll
        for (int dt = 0; dt < DH / 8; ++dt)
          *reinterpret_cast<float2*>(dst + dt * 8) = make_float2(o[mt][dt][2 * e] * f, o[mt][dt][2 * e + 1] * f);
      }
    __syncthreads();
    const bool whole = pc.whole();
    for (int u = tid; u < R * (DH / 4); u += 32 * kWarps) {
      const int r = u / (DH / 4), d = (u % (DH / 4)) * 4;
      if (t.r0 + r >= t.r1) break;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f, M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(ob + (w * R + r) * LDO + d);
        acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        L += sm_l[w * R + r];
        M = fmaxf(M, sm_m[w * R + r]);
      }
      if (whole) {
        const int tk = (t.r0 + r) / a.group, hq = h * a.group + (t.r0 + r) % a.group;
        const long long row = (long long)b * a.T + tk;
        const float inv = L == 0.f ? 0.f : a.v_scale / L;
        store4(static_cast<T*>(a.out) + row * a.os + (long long)hq * DH + d,
               make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv), a.vec);
        if (a.lse && d == 0) a.lse[row * a.n_q + hq] = kv::lse_of(M, L, a.weight_exp);
      } else {
        const size_t pr = kv::part_row(pc, R) + r;
        *reinterpret_cast<float4*>(a.part_o + pr * DH + d) = acc;
        if (d == 0) a.part_ml[pr] = make_float2(M, L);
      }
    }
    // the ring is the copies' again
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
  if (!got && lane == 0)  // let the copies in flight end (bounded) before the memory is given back
    for (int i = 0; i < PER && n_take + i < n_issue; ++i)
      tc::mbar_wait(tc::su32(full + warp + kWarps * ((n_take + i) % PER)), (uint32_t)((n_take + i) / PER) & 1u, a.status);
  if (a.stream && tid == 0) a.joins[blockIdx.x] = walk.join_of(any, pc);
}

// Joins the pieces of the segment that begins in CTA blockIdx.x's run and goes on after it: one warp per row, in order.
// Bound: two dependent loads, since nothing but their number is needed to ask for the pieces (asked for after their
// weights, eight at a time, 19 pieces of 256 rows took 2 us more).
template <typename T, int DH, int R>
__global__ void __launch_bounds__(256) kv_attention_join_kernel(const AttnArgs a) {
  pdl_trigger();
  pdl_wait();
  const int2 jn = a.joins[blockIdx.x];
  if (jn.y < 1) return;
  const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
  // piece k: slot 1 of this CTA, then slot 0 of those after it
  auto row_of = [&](int k) { return ((size_t)(blockIdx.x + k) * 2 + (k == 0)) * R + r; };
  // the first pieces' rows are asked for at once, with all else that is read
  constexpr int C = DH / 32, kAhead = 16;  // columns C lane ..
  using Part = typename std::conditional<C == 4, float4, float2>::type;
  auto part = [&](int k) { return *reinterpret_cast<const Part*>(a.part_o + row_of(k) * DH + C * lane); };
  Part ahead[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (k < jn.y) ahead[k] = part(k);
  const float2 first = lane < jn.y ? a.part_ml[row_of(lane)] : make_float2(-INFINITY, 0.f);
  const int h = jn.x % a.n_kv, j = jn.x / a.n_kv, b = j / a.row_tiles, rt = j % a.row_tiles;
  const int n = a.n_rows ? min(max(a.n_rows[b], 0), a.T) : a.T;
  if (rt * R + r >= n * a.group) return;
  float M = first.x;
  for (int k = lane + 32; k < jn.y; k += 32) M = fmaxf(M, a.part_ml[row_of(k)].x);
  M = warp_max(M);
  float L = 0.f, acc[C];
#pragma unroll
  for (int i = 0; i < C; ++i) acc[i] = 0.f;
  auto add = [&](float f, const Part& o) {
#pragma unroll
    for (int i = 0; i < C; ++i) acc[i] = fmaf(f, reinterpret_cast<const float*>(&o)[i], acc[i]);
  };
  for (int k0 = 0; k0 < jn.y; k0 += 32) {
    float w = 0.f, lw = 0.f;
    if (k0 + lane < jn.y) {
      const float2 ml = k0 ? a.part_ml[row_of(k0 + lane)] : first;
      w = ml.x == -INFINITY ? 0.f : tc::ex2_approx(ml.x - M);
      lw = w * ml.y;
    }
    L += warp_sum(lw);
    const int kn = min(32, jn.y - k0);
    if (k0 == 0)
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k < kn) add(__shfl_sync(0xffffffffu, w, k), ahead[k]);
#pragma unroll 8
    for (int k = k0 ? 0 : kAhead; k < kn; ++k) add(__shfl_sync(0xffffffffu, w, k), part(k0 + k));
  }
  const int t = (rt * R + r) / a.group, hq = h * a.group + (rt * R + r) % a.group;
  const long long row = (long long)b * a.T + t;
  const float inv = L == 0.f ? 0.f : a.v_scale / L;
  T* out = static_cast<T*>(a.out) + row * a.os + (long long)hq * DH + C * lane;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if constexpr (sizeof(T) == 4)
      out[i] = acc[i] * inv;
    else
      out[i] = __float2bfloat16_rn(acc[i] * inv);
  }
  if (a.lse && lane == 0) a.lse[row * a.n_q + hq] = kv::lse_of(M, L, a.weight_exp);
}

// A change of pieces in units: of the tcgen05 kernel in tiles of 128 keys (9,000 to 12,000 clocks against 1,100 to 1,460 a tile; 32 ragged
// requests 238 us at 4, 224 at 8, 225 at 12; 8 of 8,192 keys 20.5, 20.6, 21.3), of the other in pages (118,000 keys, 8 float32 tokens 113 us at 0,
// 108 at 8, 107 at 16, 108 at 24; 8 requests of 8,192 keys 34.1, 28.5, 28.0, 28.3; bf16 heads of 64, 32 ragged requests 208, 192, 183, 179).
constexpr int kTcChange = 8, kChange = 16;

kv::AttnPlan make_plan(const dlite_kv_attention_args& g) {
  kv::AttnPlan p;
  const int rows = g.n_q / g.cache.n_kv * g.T;
  p.tc = g.dtype == DLITE_BF16 && g.cache.d_h == 128;
  // 32-row tiles halve the conversions per row; float32 queries have twice the fragments and would spill
  p.rows = rows <= 16 || g.dtype == DLITE_F32 ? 16 : 32;
  p.row_tiles = (rows + p.rows - 1) / p.rows;
  p.unit = p.tc ? 2 : 1;
  p.change = p.tc ? kTcChange : kChange;
  // two tiles (4,000 keys, 8 tokens: 15.0 us; 20.5 with twelve; 1,000 keys: 13.3, 15.6 with four), a page for every warp
  p.min_quota = p.tc ? 2 : kWarps;
  p.grid = device_sms();            // one CTA an SM: its shared memory is the ring
  // segments that a CTA's least run holds whole are not cut
  const int most = (g.cache.max_pages + p.unit - 1) / p.unit;
  const long long tiles = (long long)g.B * p.row_tiles;
  p.stream = most > p.min_quota && tiles <= kv::kMaxList && tiles * (most + p.change) * g.cache.n_kv < (1LL << 31);
  if (!p.stream) p.grid = (int)std::min<long long>((long long)g.B * p.row_tiles * g.cache.n_kv, p.grid);
  return p;
}

int check_attention(const dlite_kv_attention_args* g) {
  if (!g || !g->q || !g->out) return DLITE_ERR_INVALID_ARG;
  const dlite_kv_cache& c = g->cache;
  if (const int rc = kv::check_cache(c, g->B, g->T, g->pos, g->n_rows, g->status)) return rc;
  if (g->dtype != DLITE_F32 && g->dtype != DLITE_BF16) return DLITE_ERR_INVALID_ARG;
  if (g->n_q < 1 || g->n_q % c.n_kv || g->window < 0 || !(g->scale > 0.f) || isinf(g->scale)) return DLITE_ERR_INVALID_ARG;
  const int es = g->dtype == DLITE_F32 ? 4 : 2;
  const long long cols = (long long)g->n_q * c.d_h;
  if (g->q_stride < cols || g->out_stride < cols || ((uintptr_t)g->q | (uintptr_t)g->out) % es || ((uintptr_t)g->lse & 3))
    return DLITE_ERR_INVALID_ARG;
  const long long rows = (long long)(g->n_q / c.n_kv) * g->T;
  if (rows > (1 << 20) || (long long)c.n_pages * c.n_kv > 0x7fffffffLL || g->B * ((rows + 15) / 16) * c.n_kv > 0x7fffffffLL)
    return DLITE_ERR_UNSUPPORTED_SHAPE;
  return DLITE_OK;
}

template <typename T, int DH, int R>
cudaError_t join(const AttnArgs& a, const kv::AttnPlan& p, cudaStream_t s) {
  if (!p.stream) return cudaSuccess;
  return launch_pdl(kv_attention_join_kernel<T, DH, R>, dim3(p.grid, R / 8), dim3(256), 0, s, a);
}
template <typename T, int DH, int MT>
cudaError_t launch(const AttnArgs& a, const kv::AttnPlan& p, cudaStream_t s) {
  using S = Shape<T, DH, MT>;
  cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<T, DH, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kv_attention_kernel<T, DH, MT>, dim3(p.grid), dim3(32 * kWarps), S::SMEM, s, a);
  return e != cudaSuccess ? e : join<T, DH, S::R>(a, p, s);
}
cudaError_t launch(const AttnArgs& a, const kv::AttnPlan& p, int d_h, int dtype, cudaStream_t s) {
  if (p.tc) {
    const cudaError_t e = kv::launch_attention_tc(a, p, s);
    return e != cudaSuccess ? e : p.rows == 16 ? join<bf16, 128, 16>(a, p, s) : join<bf16, 128, 32>(a, p, s);
  }
  if (dtype == DLITE_F32) return d_h == 128 ? launch<float, 128, 1>(a, p, s) : launch<float, 64, 1>(a, p, s);
  return p.rows == 16 ? launch<bf16, 64, 1>(a, p, s) : launch<bf16, 64, 2>(a, p, s);
}

}  // namespace
}  // namespace dlite

extern "C" size_t dlite_kv_attention_workspace(const dlite_kv_attention_args* g) {
  if (dlite::check_attention(g) != DLITE_OK) return 0;
  return dlite::make_plan(*g).bytes(g->cache.d_h);
}

extern "C" int dlite_kv_attention(const dlite_kv_attention_args* g, dlite_stream_t stream) {
  using namespace dlite;
  if (const int rc = check_attention(g)) return rc;
  const dlite_kv_cache& c = g->cache;
  const kv::AttnPlan p = make_plan(*g);
  const size_t need = p.bytes(c.d_h);
  if (need && (!g->workspace || g->workspace_bytes < need || ((uintptr_t)g->workspace & 15))) return DLITE_ERR_INVALID_ARG;
  AttnArgs a = {};
  a.pages = static_cast<const uint8_t*>(c.pages);
  a.bt = c.block_table;
  a.n_pages = c.n_pages;
  a.n_kv = c.n_kv;
  a.max_pages = c.max_pages;
  a.B = g->B;
  a.T = g->T;
  a.n_q = g->n_q;
  a.group = g->n_q / c.n_kv;
  a.row_tiles = p.row_tiles;
  a.window = g->window;
  a.unit = p.unit;
  a.min_quota = p.min_quota;
  a.change = p.change;
  a.stream = p.stream;
  a.weight_exp = p.tc ? kv::kTcWeightExp : kWeightExp;
  a.scale_mant = (float)frexp((double)g->scale * 1.4426950408889634, &a.scale_exp);
  a.scale_exp += c.k_exp;
  a.v_scale = ldexpf(1.f, c.v_exp);
  a.q = g->q;
  a.qs = g->q_stride;
  a.out = g->out;
  a.os = g->out_stride;
  a.lse = g->lse;
  a.pos = g->pos;
  a.n_rows = g->n_rows;
  a.part_o = static_cast<float*>(g->workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)p.grid * 2 * p.rows * c.d_h);
  a.joins = reinterpret_cast<int2*>(a.part_ml + (size_t)p.grid * 2 * p.rows);
  const int V = g->dtype == DLITE_F32 ? 4 : 8;
  a.vec = !(((uintptr_t)g->q | (uintptr_t)g->out) & 15) && g->q_stride % V == 0 && g->out_stride % V == 0;
  a.status = g->status;
  return launch_status(launch(a, p, c.d_h, g->dtype, (cudaStream_t)stream));
}
