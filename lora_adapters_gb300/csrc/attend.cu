// slora_kv_attend for few query rows (decode): attention of a request's new
// tokens over its paged keys and values, split over the cache's length.
//
// For a row i (one token, one query head) at position p_i
//     s_ij = c(scale q_i . k_j), j <= p_i;   o_i = sum_j e^(s_ij) v_j / sum_j e^(s_ij),
// computed in one pass with a running maximum m: the sums over any set of keys
// are (m, l = sum e^(s - m), o = sum e^(s - m) v), and two sets join as
//     m = max(m1, m2);  l = l1 e^(m1 - m) + l2 e^(m2 - m);  o likewise.
//
// Bound: memory.  Every key and value is used by heads_q / heads_kv rows only,
// 2 to 16 operations per 16-bit element, against the 280 a byte that the
// tensor cores could do.  So the kernel is built around loads:
//  - a warp takes 16 tokens of one key head at a time, K and V straight from
//    their pages into registers with 16-byte loads, the next tokens' loads in
//    flight while these are multiplied: 8 KB a warp, 12 warps an SM;
//  - the products run on warp-level tensor instructions (m16n8k16): the 16
//    tokens on M for S^T = K Q^T, the head's elements on M for O^T = V^T P^T,
//    and up to 8 rows (the query heads that share the key head) on N, so
//    neither K nor V changes lanes.  Operands come from registers; staging
//    them for the larger tensor-core shapes, 128 rows high, would leave 15/16
//    of those empty.  The order of a head's elements in the sum over d is the
//    same permutation for K and Q, chosen so that a 16-byte load is two steps'
//    operands;
//  - P is split into two 16-bit parts, hi and lo = p - hi, each its own
//    product: the weights keep twice the storage type's bits.  fp16 has few
//    exponents, so there P is 2^14 e^(s - m) (its sum alike): 22 bits for weights
//    above 2^-28 of the largest, an error of 2^-39 of it below;
//  - the work, (request, row tile, key head) x 16-token units laid end to end,
//    is cut into equal runs, one per group of warps, whatever the lengths.  A
//    run that starts or ends inside a segment leaves (m, l, o) in scratch, and
//    kv_join adds the parts of each split segment up in order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "attend.cuh"

namespace slora {
namespace {

constexpr int kDecWarps = 4;             // per CTA
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kDecCtas = 3;              // per SM: 170 registers a thread (D = 128 spills 56 to 60 bytes;
                                         // D = 256, two a SM and 255 registers, 320 to 380)

// D: head_dim rounded up to 64, 128 or 256; elements past head_dim are zeros.
template <class E, int D, bool CAP>
__global__ void __launch_bounds__(kDecThreads, D <= 128 ? kDecCtas : 2)
kv_decode_kernel(const __grid_constant__ KvAttendArgs a) {
  constexpr int NB = D / 64;        // 64-element blocks of a head (V)
  constexpr int NC = D / 32;        // 32-element chunks of a head (K, Q)
  constexpr float kUp = Elem<E>::kBf16 ? 0.f : 14.f;   // weights are held times 2^kUp
  const KvDev& d = a.kv;
  const int tid = threadIdx.x, lane = tid & 31;
  const int hbw = a.hbw, blocks = d.heads_kv / hbw;
  const int64_t gw = (int64_t)blockIdx.x * kDecWarps + (tid >> 5);
  const int64_t groups = (int64_t)gridDim.x * kDecWarps / hbw;
  const DecSplit sp = dec_split(__ldg(d.dec_off + a.R), blocks, groups);
  const int64_t g = gw / hbw;
  int64_t u = g * sp.run;
  const int64_t u1 = min(sp.total, u + sp.run);
  const int hsub = (int)(gw - g * hbw);

  const int dim = d.head_dim, P = d.per_page, group = d.heads_q / d.heads_kv;
  const int kk = lane & 3, nn = lane >> 2;
  const int64_t row_bytes = (int64_t)d.heads_kv * dim * 2;
  const int64_t plane = (int64_t)d.max_rows * d.max_blocks;
  const float sc = kLog2e * a.scale, cap_t = a.cap_t, cap2 = a.cap2;
  if (u >= u1) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  int left = (int)min(u1 - u, (int64_t)0x7fffffff);     // units to do (a run of more than 2^31 units has no cache to be in)

  // The units to do are fetched two ahead of the one that is multiplied, from
  // one segment into the next: `f` is where that is.
  struct {
    int left, r, hb, rt, c;        // units left; request, head block, row tile, unit of the segment
    int n, tiles, len;             // units of a segment, row tiles, tokens of the request
    int at;                        // byte of a pool row at which the head block's head of this warp starts
    const int32_t* tab;            // lanes 0-15 the request's K pages, 16-31 its V pages
  } f;
  auto f_open = [&](const int4& rq) {
    f.len = rq.z;
    f.n = (rq.z + kKvUnit - 1) / kKvUnit;
    f.tiles = (rq.y * group + kKvRowTile - 1) / kKvRowTile;
    f.tab = d.table + (2 * a.layer + (lane >> 4)) * plane + (int64_t)dbg_index(rq.w, d.max_rows, d.error) * d.max_blocks;
  };
  // requests without units here: no new tokens, or a chunk
  auto no_units = [&](const int4& rq) {
    return rq.y == 0 || (a.tpt > 0 && (int64_t)rq.y * group > kKvChunkRows);
  };
  {
    f.left = left;
    f.r = find_request(d.dec_off, a.R, u, blocks);
    const int4 rq = __ldg(d.req + f.r);
    f_open(rq);
    const int64_t in_req = u - (int64_t)__ldg(d.dec_off + f.r) * blocks;
    const int seg = (int)(in_req / f.n);
    f.c = (int)(in_req - (int64_t)seg * f.n);
    f.hb = seg / f.tiles;
    f.rt = seg - f.hb * f.tiles;
    f.at = (f.hb * hbw + hsub) * dim * 2;
  }
  int r = f.r, hb = f.hb, rt = f.rt, c0 = f.c;          // the segment that is multiplied
  // The next unit's pool rows, one a lane (-1: past the request's length, kNoPage:
  // no such page), and where its head starts in them.
  constexpr int kNoPage = -2;
  auto fetch = [&](int& at) -> int {
    if (f.left == 0) return -1;
    --f.left;
    if (f.c == f.n) {
      f.c = 0;
      if (++f.rt == f.tiles) {
        f.rt = 0;
        if (++f.hb == blocks) {
          f.hb = 0;
          int4 rq;
          do rq = __ldg(d.req + ++f.r);
          while (no_units(rq));
          f_open(rq);
        }
        f.at = (f.hb * hbw + hsub) * dim * 2;
      }
    }
    at = f.at;
    const int j = f.c++ * kKvUnit + (lane & 15);
    if (j >= f.len) return -1;
    const int b = (int)a.per_page_div.div((uint32_t)j);
    const int page = __ldg(f.tab + b);
    return (uint32_t)page < (uint32_t)d.num_pages ? page * P + (j - b * P) : kNoPage;
  };
  uint4 kf[NC][2], vf[NB][4];
  auto load_k = [&](int slot, int at) {
    const uint8_t* base = reinterpret_cast<const uint8_t*>(d.pool) + (at + kk * 16);
    const int s0 = __shfl_sync(0xffffffffu, slot, nn), s1 = __shfl_sync(0xffffffffu, slot, nn + 8);
    const uint8_t* p0 = base + s0 * row_bytes;
    const uint8_t* p1 = base + s1 * row_bytes;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const bool in = D == dim || (i * 4 + kk) * 8 < dim;
      kf[i][0] = in && s0 >= 0 ? load_stream(p0 + i * 64) : make_uint4(0, 0, 0, 0);
      kf[i][1] = in && s1 >= 0 ? load_stream(p1 + i * 64) : make_uint4(0, 0, 0, 0);
    }
  };
  auto load_v = [&](int slot, int at) {
    const uint8_t* base = reinterpret_cast<const uint8_t*>(d.pool) + (at + nn * 16);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int s = __shfl_sync(0xffffffffu, slot, 16 + 2 * kk + (x & 1) + (x & 2) * 4);
      const uint8_t* p = base + s * row_bytes;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const bool in = D == dim || b * 64 + nn * 8 < dim;
        vf[b][x] = in && s >= 0 ? load_stream(p + b * 128) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  int at = 0, at_next = 0, lowest = 0;
  int slot = fetch(at), slot_next = fetch(at_next);
  load_k(slot, at);
  load_v(slot, at);

  while (left > 0) {
    int4 rq = __ldg(d.req + r);
    while (no_units(rq)) rq = __ldg(d.req + ++r);
    const int len = rq.z, q0 = rq.x, rows = rq.y * group;
    const int nchunk = (len + kKvUnit - 1) / kKvUnit, tiles = (rows + kKvRowTile - 1) / kKvRowTile;
    const int c1 = min(nchunk, c0 + left);
    const int hk = hb * hbw + hsub;
    const int ctx = len - rq.y;
    // ---- this tile's queries: row n of the tile is (token, head of the group)
    uint32_t qf[NC][4];
    {
      const int row = rt * kKvRowTile + nn;
      const bool in = row < rows;
      const uint16_t* src = a.q + (int64_t)dbg_index(q0 + (in ? row / group : 0), a.T, d.error) * a.ldq +
                            (int64_t)(hk * group + (in ? row % group : 0)) * dim;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int e = (i * 4 + kk) * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (in && e < dim) v = *reinterpret_cast<const uint4*>(src + e);
        qf[i][0] = v.x; qf[i][1] = v.y; qf[i][2] = v.z; qf[i][3] = v.w;
      }
    }
    // keys row 2 kk (+ 1) may see: positions below lim0 (lim1)
    const int last = rows - 1;
    const int lim0 = ctx + min(rt * kKvRowTile + 2 * kk, last) / group + 1;
    const int lim1 = ctx + min(rt * kKvRowTile + 2 * kk + 1, last) / group + 1;

    float o[4 * NB][4];
#pragma unroll
    for (int i = 0; i < 4 * NB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    for (int c = c0; c < c1; ++c) {
      // S^T: tokens nn and nn + 8, rows 2 kk and 2 kk + 1
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        mma16816<E>(s, kf[i][0].x, kf[i][1].x, kf[i][0].y, kf[i][1].y, qf[i][0], qf[i][1]);
        mma16816<E>(s, kf[i][0].z, kf[i][1].z, kf[i][0].w, kf[i][1].w, qf[i][2], qf[i][3]);
      }
      const int held = slot;
      slot = slot_next;
      at = at_next;
      slot_next = fetch(at_next);
      load_k(slot, at);
      // a token without a K or a V row has no weight
      const uint32_t none = __ballot_sync(0xffffffffu, held < 0), gone = (none | none >> 16) >> nn;
      const bool v0 = !(gone & 1), v1 = !(gone >> 8 & 1);
      lowest = min(lowest, held);
      const int j0 = c * 16 + nn, j1 = j0 + 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = CAP ? capped<true>(s[i], sc, cap_t, cap2) : s[i] * sc;
        const bool seen = (i & 2 ? v1 : v0) && (i & 2 ? j1 : j0) < (i & 1 ? lim1 : lim0);
        s[i] = seen ? x : -INFINITY;
      }
      float n0 = fmaxf(s[0], s[2]), n1 = fmaxf(s[1], s[3]);
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, x));
        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, x));
      }
      n0 = fmaxf(n0, m0);
      n1 = fmaxf(n1, m1);
      if (__any_sync(0xffffffffu, n0 != m0 || n1 != m1)) {
        const float f0 = n0 == m0 ? 1.f : ex2(m0 - n0), f1 = n1 == m1 ? 1.f : ex2(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int i = 0; i < 4 * NB; ++i) {
          o[i][0] *= f0; o[i][1] *= f1; o[i][2] *= f0; o[i][3] *= f1;
        }
      }
      // a row that has seen no key yet has m = -inf; its weights are zeros
      const float z0 = m0 == -INFINITY ? 0.f : m0 - kUp, z1 = m1 == -INFINITY ? 0.f : m1 - kUp;
      const float p0 = ex2(s[0] - z0), p1 = ex2(s[1] - z1), p2 = ex2(s[2] - z0), p3 = ex2(s[3] - z1);
      l0 += p0 + p2;
      l1 += p1 + p3;
      const uint32_t ha = Elem<E>::from2(p0, p1), hb2 = Elem<E>::from2(p2, p3);
      const float2 fa = Elem<E>::to2(ha), fb = Elem<E>::to2(hb2);
      const uint32_t h0 = trans8x8(ha), h1 = trans8x8(hb2);
      const uint32_t e0 = trans8x8(Elem<E>::from2(p0 - fa.x, p1 - fa.y)),
                     e1 = trans8x8(Elem<E>::from2(p2 - fb.x, p3 - fb.y));
      // O^T: element pairs of V's 16-byte pieces on M, two tokens a register
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t* w0 = &vf[b][0].x;
        const uint32_t* w1 = &vf[b][1].x;
        const uint32_t* w2 = &vf[b][2].x;
        const uint32_t* w3 = &vf[b][3].x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a0 = __byte_perm(w0[j], w1[j], 0x5410), a1 = __byte_perm(w0[j], w1[j], 0x7632);
          const uint32_t a2 = __byte_perm(w2[j], w3[j], 0x5410), a3 = __byte_perm(w2[j], w3[j], 0x7632);
          mma16816<E>(o[b * 4 + j], a0, a1, a2, a3, h0, h1);
          mma16816<E>(o[b * 4 + j], a0, a1, a2, a3, e0, e1);
        }
      }
      load_v(slot, at);
    }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, x);
      l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
    // ---- rows 2 kk and 2 kk + 1, elements 64 b + 8 nn .. + 7
    const bool whole = c0 == 0 && c1 == nchunk;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = rt * kKvRowTile + 2 * kk + x;
      if (row >= rows) continue;
      const float l = x ? l1 : l0;
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* dst = a.out + (int64_t)dbg_index(q0 + row / group, a.T, d.error) * a.ldo +
                        (int64_t)(hk * group + row % group) * dim + nn * 8;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float y[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            y[2 * j] = o[b * 4 + j][x] * inv;
            y[2 * j + 1] = o[b * 4 + j][2 + x] * inv;
          }
          if (D == dim || b * 64 + nn * 8 < dim) *reinterpret_cast<uint4*>(dst + b * 64) = pack8<E>(y);
        }
      } else {
        // slot 0: the segment began in an earlier run; slot 1: it begins here
        const int64_t part = (gw * 2 + (c0 == 0 ? 1 : 0)) * kKvRowTile + 2 * kk + x;
        float* dst = a.part_o + part * D + nn * 8;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          *reinterpret_cast<float4*>(dst + b * 64) =
              make_float4(o[b * 4][x], o[b * 4][2 + x], o[b * 4 + 1][x], o[b * 4 + 1][2 + x]);
          *reinterpret_cast<float4*>(dst + b * 64 + 4) =
              make_float4(o[b * 4 + 2][x], o[b * 4 + 2][2 + x], o[b * 4 + 3][x], o[b * 4 + 3][2 + x]);
        }
        if (nn == 0) a.part_ml[part] = make_float2(x ? m1 : m0, l);
      }
    }
    left -= c1 - c0;
    c0 = 0;                        // the next segment, if any is left
    if (++rt == tiles) {
      rt = 0;
      if (++hb == blocks) {
        hb = 0;
        ++r;
      }
    }
  }
  if (lowest == kNoPage) report_err(d.error, kErrInvalid);
  // after chunks: their kernel may still run, and this grid ends after it
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The parts of the split segments, joined in the order of the cache.  Decode:
// an item is one row (request, token, query head); where it was split follows
// from the same sums the decode kernel divides its work by.  A warp per item;
// with few requests, whose segments have many parts each, a block per item,
// its warps taking every so-many-th part.  Chunks: a warp per row.
constexpr int kJoinThreads = 256;
constexpr int kJoinWideWarps = 16;

// NORMED: the parts' o are divided by their l already, and so is the sum (4-bit caches, whose
// values reach 2^127 in bf16: sums of them over a part's tokens would not be finite).
template <int V, bool NORMED = false>
struct JoinSum {
  float m = -INFINITY, l = 0.f, o[V] = {};
  // (a part without weight: its sums may not have been written.  m = -inf alone does
  // not say so: scores that are not numbers leave it there, and l is not a number)
  __device__ __forceinline__ void add(float2 ml, const float (&y)[V]) {
    if (ml.y == 0.f) return;
    const float mn = fmaxf(m, ml.x), f = ex2(m - mn), w = ex2(ml.x - mn);
    m = mn;
    if constexpr (NORMED) {
      const float a = l * f, b = ml.y * w;
      l = a + b;
      const float fo = a / l, wo = b / l;
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = o[j] * fo + y[j] * wo;
    } else {
      l = l * f + ml.y * w;
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = o[j] * f + y[j] * w;
    }
  }
};
// A lane's elements of a row of `cols` floats: 4 consecutive ones of every 128
// (2 of 64), as floats j of y.
template <int V>
__device__ __forceinline__ void load_row(const float* row, int lane, float (&y)[V]) {
  if constexpr (V == 2) {
    const float2 v = __ldcg(reinterpret_cast<const float2*>(row) + lane);
    y[0] = v.x; y[1] = v.y;
  } else {
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(row + j * 128) + lane);
      y[4 * j] = v.x; y[4 * j + 1] = v.y; y[4 * j + 2] = v.z; y[4 * j + 3] = v.w;
    }
  }
}
template <class E, int V>
__device__ __forceinline__ void store_row(uint16_t* row, int lane, int dim, const float (&o)[V], float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if constexpr (V == 2) {
    if (lane * 2 < dim) *reinterpret_cast<uint32_t*>(row + lane * 2) = Elem<E>::from2(o[0] * inv, o[1] * inv);
  } else {
#pragma unroll
    for (int j = 0; j < V / 4; ++j)
      if (j * 128 + lane * 4 < dim)
        *reinterpret_cast<uint2*>(row + j * 128 + lane * 4) =
            make_uint2(Elem<E>::from2(o[4 * j] * inv, o[4 * j + 1] * inv),
                       Elem<E>::from2(o[4 * j + 2] * inv, o[4 * j + 3] * inv));
  }
}

template <class E, int D, bool WIDE, bool NORMED>
__global__ void __launch_bounds__(WIDE ? kJoinWideWarps * 32 : kJoinThreads)
kv_join_kernel(const __grid_constant__ KvAttendArgs a, const int64_t groups) {
  constexpr int V = D / 32;      // elements per lane
  constexpr int W = WIDE ? kJoinWideWarps : 1;
  __shared__ float s_o[W][D];
  __shared__ float s_f[W], s_m[W], s_l[W];
  const KvDev& d = a.kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hbw = a.hbw, blocks = d.heads_kv / hbw, group = d.heads_q / d.heads_kv, dim = d.head_dim;
  const DecSplit sp = dec_split(__ldg(d.dec_off + a.R), blocks, groups);
  // what the plan says about the first item is read while the decode kernel
  // still runs; its parts are read after it, and no block leaves before it
  bool waited = false;
  // items: request, row, key head (fastest)
  const int per_req = a.rows * d.heads_kv;
  const int64_t items = (int64_t)a.R * per_req, stride = (int64_t)gridDim.x * (WIDE ? 1 : blockDim.x / 32);
  for (int64_t it = WIDE ? blockIdx.x : (int64_t)blockIdx.x * (blockDim.x / 32) + warp; it < items; it += stride) {
    const int r = (int)(it / per_req), in = (int)(it - (int64_t)r * per_req), row = in / d.heads_kv,
              hk = in - row * d.heads_kv;
    const int4 rq = __ldg(d.req + r);
    const int off = __ldg(d.dec_off + r), off_next = __ldg(d.dec_off + r + 1);
    const int rows = rq.y * group;
    if (row >= rows || off == off_next) continue;         // no such row, or a chunk
    const int nchunk = (rq.z + d.unit - 1) >> (31 - __clz(d.unit)), tiles = (rows + a.row_tile - 1) / a.row_tile, rt = row / a.row_tile,
              n = row - rt * a.row_tile;
    const int hb = hk / hbw, hsub = hk - hb * hbw;
    const int64_t us = (int64_t)off * blocks + (int64_t)(hb * tiles + rt) * nchunk;
    const int64_t g0 = us / sp.run, g1 = (us + nchunk - 1) / sp.run;
    if (g0 == g1) continue;                               // the decode kernel wrote it
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
    waited = true;
    JoinSum<V, NORMED> s;
    for (int64_t g = g0 + (WIDE ? warp : 0); g <= g1; g += 4 * W) {   // four parts on their way at a time
      float2 ml[4];
      float y[4][V];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        const int64_t gk = g + k * W;
        if (gk <= g1) {
          const int64_t part = ((gk * hbw + hsub) * 2 + (gk == g0 ? 1 : 0)) * kKvRowTile + n;
          ml[k] = __ldcg(a.part_ml + part);
          load_row<V>(a.part_o + part * D, lane, y[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) s.add(ml[k], y[k]);
    }
    uint16_t* dst = a.out + (int64_t)dbg_index(rq.x + row / group, a.T, d.error) * a.ldo +
                    (int64_t)(hk * group + row % group) * dim;
    if constexpr (!WIDE) {
      store_row<E, V>(dst, lane, dim, s.o, NORMED && s.l != 0.f ? 1.f : s.l);
    } else {                                              // the warps' sums, in their order
#pragma unroll
      for (int j = 0; j < V; ++j) s_o[warp][j * 32 + lane] = s.o[j];
      if (lane == 0) {
        s_m[warp] = s.m;
        s_l[warp] = s.l;
      }
      __syncthreads();
      if (warp == 0) {
        float m = lane < W ? s_m[lane] : -INFINITY;
        const float own = m;
#pragma unroll
        for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        if (lane < W) s_f[lane] = ex2(own - m);
        __syncwarp();
        float l = 0.f, y[V] = {};
        if (NORMED)
          for (int k = 0; k < W; ++k) l += s_l[k] == 0.f ? 0.f : s_l[k] * s_f[k];
        const float all = l;
#pragma unroll 4
        for (int k = 0; k < W; ++k) {
          if (s_l[k] == 0.f) continue;                    // no weight
          const float f = NORMED ? s_l[k] * s_f[k] / all : s_f[k];
          if (!NORMED) l += s_l[k] * f;
#pragma unroll
          for (int j = 0; j < V; ++j) y[j] += s_o[k][j * 32 + lane] * f;
        }
        store_row<E, V>(dst, lane, dim, y, NORMED && l != 0.f ? 1.f : l);
      }
      __syncthreads();
    }
  }
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Rows are spread over gridDim.y blocks of every CTA's split segment.
constexpr int kChunkJoinThreads = 256;
template <class E>
__global__ void __launch_bounds__(kChunkJoinThreads) kv_chunk_join_kernel(const __grid_constant__ KvAttendArgs a) {
  const KvDev& d = a.kv;
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int first = blockIdx.x;
  const int4 sg = __ldcg(a.tc_split + first);
  if (sg.x < 0) return;
  const int group = d.heads_q / d.heads_kv, dim = d.head_dim, rows_a = (sg.y >> 16) * group,
            rows = rows_a + (sg.y & 0xffff) * group;
  for (int row = blockIdx.y * (kChunkJoinThreads / 32) + (threadIdx.x >> 5); row < rows;
       row += gridDim.y * (kChunkJoinThreads / 32)) {
    const int x = row >= rows_a, rho = row - (x ? rows_a : 0), tok = rho / group;
    JoinSum<4> s;
    for (int g = first; g <= sg.w; g += 4) {
      float2 ml[4];
      float y[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        if (g + k <= sg.w) {
          const int64_t part = (((int64_t)(g + k) * 2 + (g + k == first ? 1 : 0)) * 2 + x) * kKvTile + rho;
          ml[k] = __ldcg(a.tc_part_ml + part);
          load_row<4>(a.tc_part_o + part * kKvTile, lane, y[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) s.add(ml[k], y[k]);
    }
    store_row<E, 4>(a.out + (int64_t)dbg_index(sg.x + x * a.tpt + tok, a.T, d.error) * a.ldo +
                        (int64_t)(sg.z * group + rho - tok * group) * dim,
                    lane, dim, s.o, s.l);
  }
}

// `groups`: the groups of warps that the decode kernel shared the work out to.
template <class E, int D, bool NORMED>
cudaError_t launch_join(const KvAttendArgs& a, int num_sms, bool after_chunks, int64_t groups, cudaStream_t st) {
  if (after_chunks) {
    const cudaError_t e = launch_early(kv_chunk_join_kernel<E>, dim3(num_sms, 16), kChunkJoinThreads, 0, st, a);
    if (e != cudaSuccess) return e;
  }
  const int64_t items = (int64_t)a.R * a.rows * a.kv.heads_kv;
  // segments of 16 parts or more on average: a block each (a 131072-token
  // context, 228 parts a row: 24 us with a warp each, 8 with a block)
  const int64_t segments = (int64_t)a.R * ((a.rows + a.row_tile - 1) / a.row_tile) * (a.kv.heads_kv / a.hbw);
  if (segments * 16 <= groups)
    return launch_early(kv_join_kernel<E, D, true, NORMED>, dim3((unsigned)std::min<int64_t>(items, 16 * num_sms)),
                        kJoinWideWarps * 32, 0, st, a, groups);
  const int64_t ctas = (items + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  return launch_early(kv_join_kernel<E, D, false, NORMED>, dim3((unsigned)std::min<int64_t>(ctas, 16 * num_sms)), kJoinThreads, 0,
                      st, a, groups);
}

template <class E, int D>
cudaError_t launch_decode(const KvAttendArgs& a, int num_sms, bool after_chunks, cudaStream_t st) {
  const int grid = num_sms * (D <= 128 ? kDecCtas : 2);
  auto kernel = a.softcap > 0.f ? kv_decode_kernel<E, D, true> : kv_decode_kernel<E, D, false>;
  cudaError_t e;
  if (after_chunks) {
    e = launch_early(kernel, dim3(grid), kDecThreads, 0, st, a);
  } else {
    kernel<<<grid, kDecThreads, 0, st>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  return launch_join<E, D, false>(a, num_sms, after_chunks, (int64_t)grid * kDecWarps / a.hbw, st);
}

template <class E>
cudaError_t decode_dispatch(const KvAttendArgs& a, int num_sms, bool after_chunks, cudaStream_t st) {
  if (a.kv.head_dim <= 64) return launch_decode<E, 64>(a, num_sms, after_chunks, st);
  if (a.kv.head_dim <= 128) return launch_decode<E, 128>(a, num_sms, after_chunks, st);
  return launch_decode<E, 256>(a, num_sms, after_chunks, st);
}

template <class E>
cudaError_t normed_join(const KvAttendArgs& a, int num_sms, bool after_chunks, int64_t groups, cudaStream_t st) {
  if (a.kv.head_dim <= 64) return launch_join<E, 64, true>(a, num_sms, after_chunks, groups, st);
  if (a.kv.head_dim <= 128) return launch_join<E, 128, true>(a, num_sms, after_chunks, groups, st);
  return launch_join<E, 256, true>(a, num_sms, after_chunks, groups, st);
}
}  // namespace

static_assert(kDecCtas * kDecWarps <= kKvDecodeWarps, "the scratch has room for every warp's parts");
int64_t kv_attend_parts(int num_sms) { return (int64_t)num_sms * kKvDecodeWarps * 2 * kKvRowTile; }
int32_t kv_attend_cols(int32_t head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

template <class E, int D>
cudaError_t prepare_decode() {
  // all of the SM's memory as first-level cache, which holds the loads in flight
  // (left to itself the kernel inherits the chunk kernel's split on its SMs)
  for (auto k : {kv_decode_kernel<E, D, false>, kv_decode_kernel<E, D, true>})
    if (cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxL1))
      return e;
  return cudaSuccess;
}
cudaError_t prepare_kv_decode_kernels() {
  for (auto f : {prepare_decode<__half, 64>, prepare_decode<__half, 128>, prepare_decode<__half, 256>,
                 prepare_decode<__nv_bfloat16, 64>, prepare_decode<__nv_bfloat16, 128>, prepare_decode<__nv_bfloat16, 256>})
    if (cudaError_t e = f()) return e;
  return cudaSuccess;
}

cudaError_t launch_kv_q4_join(const KvAttendArgs& a, int dtype, int num_sms, bool after_chunks, int64_t groups,
                           cudaStream_t st) {
  return dtype == 0 ? normed_join<__half>(a, num_sms, after_chunks, groups, st)
                    : normed_join<__nv_bfloat16>(a, num_sms, after_chunks, groups, st);
}

cudaError_t launch_kv_decode(const KvAttendArgs& args, int dtype, int num_sms, bool after_chunks, cudaStream_t st) {
  KvAttendArgs a = args;
  // Warps that work side by side on neighbouring heads of the same tokens, so
  // that what they read of a page at about the same time is long: the largest
  // power of two up to 16 that divides the key heads (256 requests, 32 key
  // heads of 128: 334 us with 1, 257 with 4, 247 with 8, 243 with 16, 247
  // with 32; 8 key heads: 367, 352 and 350 us with 1, 4 and 8).
  a.hbw = heads_abreast(a.kv.heads_kv);
  return dtype == 0 ? decode_dispatch<__half>(a, num_sms, after_chunks, st)
                    : decode_dispatch<__nv_bfloat16>(a, num_sms, after_chunks, st);
}

}  // namespace slora
