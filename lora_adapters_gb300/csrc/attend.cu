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
//    product: the weights keep twice the storage type's bits;
//  - the work, (request, row tile, key head) x 16-token units laid end to end,
//    is cut into equal runs, one per group of warps, whatever the lengths.  A
//    run that starts or ends inside a segment leaves (m, l, o) in scratch, and
//    kv_join adds the parts of each split segment up in order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "kv.cuh"
#include "kv.h"

namespace slora {
namespace {

constexpr int kDecWarps = 4;             // per CTA
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kDecCtas = 3;              // per SM: 170 registers a thread
constexpr int kDecMinUnits = 2;          // shortest run: 32 tokens
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Streaming 16-byte load: every byte of the cache is used once per call.
__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
template <class E>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (Elem<E>::kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8x8 matrix of 16-bit elements held as one packed pair a lane.
__device__ __forceinline__ uint32_t trans8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The units of a call: segment = (request, row tile of kKvRowTile rows, block
// of `hbw` key heads), ceil(len / 16) units each, laid out request by request.
struct DecSplit {
  int64_t total;     // units
  int64_t run;       // units per group of warps
};
__device__ __forceinline__ DecSplit dec_split(int units, int blocks, int64_t groups) {
  DecSplit s;
  s.total = (int64_t)units * blocks;
  s.run = max((int64_t)kDecMinUnits, (s.total + groups - 1) / groups);
  return s;
}
// Largest r with off[r] <= x.
__device__ __forceinline__ int find_request(const int32_t* off, int R, int64_t x, int blocks) {
  int lo = 0, hi = R - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int64_t)off[mid] * blocks <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// D: head_dim rounded up to 64, 128 or 256; elements past head_dim are zeros.
template <class E, int D, bool CAP>
__global__ void __launch_bounds__(kDecThreads, D <= 128 ? kDecCtas : 2)
kv_decode_kernel(const __grid_constant__ KvAttendArgs a) {
  constexpr int NB = D / 64;        // 64-element blocks of a head (V)
  constexpr int NC = D / 32;        // 32-element chunks of a head (K, Q)
  __shared__ int32_t off[kKvMaxRequests + 1];
  const KvDev& d = a.kv;
  const int tid = threadIdx.x, lane = tid & 31;
  for (int i = tid; i <= a.R; i += kDecThreads) off[i] = d.dec_off[i];
  __syncthreads();
  const int hbw = a.hbw, blocks = d.heads_kv / hbw;
  const int64_t gw = (int64_t)blockIdx.x * kDecWarps + (tid >> 5);
  const int64_t groups = (int64_t)gridDim.x * kDecWarps / hbw;
  const DecSplit sp = dec_split(off[a.R], blocks, groups);
  const int64_t g = gw / hbw;
  int64_t u = g * sp.run;
  const int64_t u1 = min(sp.total, u + sp.run);
  if (u >= u1) return;
  const int hsub = (int)(gw - g * hbw);

  const int dim = d.head_dim, P = d.per_page, group = d.heads_q / d.heads_kv;
  const int kk = lane & 3, nn = lane >> 2;
  const int64_t row_bytes = (int64_t)d.heads_kv * dim * 2;
  const int64_t plane = (int64_t)d.max_rows * d.max_blocks;
  const float sc = CAP ? 2.f * kLog2e * a.scale / a.softcap : kLog2e * a.scale;
  const float cap2 = a.softcap * kLog2e;
  int r = find_request(off, a.R, u, blocks);

  while (u < u1) {
    while ((int64_t)off[r + 1] * blocks <= u) ++r;      // requests without units are passed over
    const int len = d.kv_len[r], q0 = d.q_start[r], rows = (d.q_start[r + 1] - q0) * group;
    const int nchunk = (len + 15) >> 4, tiles = (rows + kKvRowTile - 1) / kKvRowTile;
    const int64_t in_req = u - (int64_t)off[r] * blocks;
    const int seg = (int)(in_req / nchunk), c0 = (int)(in_req - (int64_t)seg * nchunk);
    const int hb = seg / tiles, rt = seg - hb * tiles;
    const int c1 = (int)min((int64_t)nchunk, c0 + (u1 - u));
    const int hk = hb * hbw + hsub;
    const int ctx = len - rows / group;
    // ---- this tile's queries: row n of the tile is (token, head of the group)
    uint32_t qf[NC][4];
    {
      const int row = rt * kKvRowTile + nn;
      const bool in = row < rows;
      const uint16_t* src = a.q + (int64_t)(q0 + (in ? row / group : 0)) * a.ldq +
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

    // lanes 0-15 look up the K rows of a unit's tokens, lanes 16-31 the V rows
    const int32_t* tab = d.table + (2 * a.layer + (lane >> 4)) * plane + (int64_t)d.row[r] * d.max_blocks;
    auto lookup = [&](int c) -> int {
      const int j = c * 16 + (lane & 15);
      if (c >= c1 || j >= len) return -1;
      const int b = (int)a.per_page_div.div((uint32_t)j);
      const int page = __ldg(tab + b);
      return (uint32_t)page < (uint32_t)d.num_pages ? page * P + (j - b * P) : -1;
    };
    const uint8_t* base = reinterpret_cast<const uint8_t*>(d.pool) + (int64_t)hk * dim * 2;
    uint4 kf[NC][2], vf[NB][4];
    auto load_k = [&](int slot) {
      const int s0 = __shfl_sync(0xffffffffu, slot, nn), s1 = __shfl_sync(0xffffffffu, slot, nn + 8);
      const uint8_t* p0 = base + s0 * row_bytes + kk * 16;
      const uint8_t* p1 = base + s1 * row_bytes + kk * 16;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const bool in = D == dim || (i * 4 + kk) * 8 < dim;
        kf[i][0] = in && s0 >= 0 ? load_stream(p0 + i * 64) : make_uint4(0, 0, 0, 0);
        kf[i][1] = in && s1 >= 0 ? load_stream(p1 + i * 64) : make_uint4(0, 0, 0, 0);
      }
    };
    auto load_v = [&](int slot) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int s = __shfl_sync(0xffffffffu, slot, 16 + 2 * kk + (x & 1) + (x & 2) * 4);
        const uint8_t* p = base + s * row_bytes + nn * 16;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const bool in = D == dim || b * 64 + nn * 8 < dim;
          vf[b][x] = in && s >= 0 ? load_stream(p + b * 128) : make_uint4(0, 0, 0, 0);
        }
      }
    };

    int slot = lookup(c0), slot_next = lookup(c0 + 1);
    load_k(slot);
    load_v(slot);
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
      slot_next = lookup(c + 2);
      load_k(slot);
      const bool v0 = __shfl_sync(0xffffffffu, held, nn) >= 0, v1 = __shfl_sync(0xffffffffu, held, nn + 8) >= 0;
      const int j0 = c * 16 + nn, j1 = j0 + 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x = s[i] * sc;
        if (CAP) x = cap2 - 2.f * cap2 * __frcp_rn(1.f + ex2(x));   // cap tanh(.), in powers of two
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
      const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
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
      load_v(slot);
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
        const float inv = l > 0.f ? 1.f / l : 0.f;
        uint16_t* dst = a.out + (int64_t)(q0 + row / group) * a.ldo + (int64_t)(hk * group + row % group) * dim + nn * 8;
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
    u += c1 - c0;
  }
}

// The parts of every split segment added up, in the order of the cache.  Every
// CTA lists the split segments for itself (each thread looks at some of the
// borders between runs), then takes (segment, head, row) items; its warps take
// every kJoinWarps-th part, and the warps' sums are added in warp order.
struct JoinItem {
  int32_t r, seg;        // request; block of heads * tiles + row tile
  int32_t first, last;   // groups of warps that hold its parts
};
constexpr int kJoinList = 512;      // borders looked at per round

template <class E, int D>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(const __grid_constant__ KvAttendArgs a,
                                                               const int64_t groups) {
  constexpr int V = D / 32;      // elements per lane
  __shared__ int32_t off[kKvMaxRequests + 1];
  __shared__ JoinItem items[kJoinList];
  __shared__ int32_t start[kJoinList + 1];     // first (head, row) item of each listed segment
  __shared__ int32_t warp_n[kJoinWarps];
  __shared__ __align__(16) float s_o[kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  const KvDev& d = a.kv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i <= a.R; i += kJoinThreads) off[i] = d.dec_off[i];
  __syncthreads();
  const int hbw = a.hbw, blocks = d.heads_kv / hbw, group = d.heads_q / d.heads_kv, dim = d.head_dim;
  const DecSplit sp = dec_split(off[a.R], blocks, groups);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t borders = (sp.total + sp.run - 1) / sp.run - 1;    // run g + 1 starts at (g + 1) * sp.run
  for (int64_t b0 = 0; b0 < borders; b0 += kJoinList) {
    // ---- list: a segment is listed by the first border inside it
    __syncthreads();
    for (int i = tid; i < kJoinList; i += kJoinThreads) {
      JoinItem it{-1, 0, 0, 0};
      const int64_t g = b0 + i + 1;
      if (g <= borders) {
        const int64_t u = g * sp.run;
        int r = find_request(off, a.R, u, blocks);
        while ((int64_t)off[r + 1] * blocks <= u) ++r;
        const int nchunk = (d.kv_len[r] + 15) >> 4;
        const int64_t in_req = u - (int64_t)off[r] * blocks;
        const int seg = (int)(in_req / nchunk);
        const int64_t us = (int64_t)off[r] * blocks + (int64_t)seg * nchunk;
        if (us < u && (g - 1) * sp.run <= us)
          it = JoinItem{r, seg, (int32_t)(g - 1), (int32_t)((us + nchunk - 1) / sp.run)};
      }
      items[i] = it;
      int n = 0;
      if (it.r >= 0) {
        const int rows = (d.q_start[it.r + 1] - d.q_start[it.r]) * group;
        const int tiles = (rows + kKvRowTile - 1) / kKvRowTile;
        n = hbw * min(kKvRowTile, rows - (it.seg % tiles) * kKvRowTile);
      }
      start[i] = n;
    }
    __syncthreads();
    if (warp == 0) {       // exclusive sums of the item counts
      int run = 0;
      for (int i = lane; i < kJoinList; i += 32) {
        const int n = start[i];
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        start[i] = run + inc - n;
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) start[kJoinList] = run;
    }
    __syncthreads();
    const int total = start[kJoinList];
    for (int x = blockIdx.x; x < total; x += gridDim.x) {
      int lo = 0, hi = kJoinList - 1;          // the last segment that starts at or before x
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= x) lo = mid;
        else hi = mid - 1;
      }
      const JoinItem it = items[lo];
      const int q0 = d.q_start[it.r], rows = (d.q_start[it.r + 1] - q0) * group;
      const int tiles = (rows + kKvRowTile - 1) / kKvRowTile;
      const int rt = it.seg % tiles, hsub = (x - start[lo]) % hbw, n = (x - start[lo]) / hbw;
      const int hk = (it.seg / tiles) * hbw + hsub, row = rt * kKvRowTile + n;
      float m = -INFINITY, l = 0.f;
      alignas(16) float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = 0.f;
#pragma unroll 4
      for (int g = it.first + warp; g <= it.last; g += kJoinWarps) {
        const int64_t part = (((int64_t)g * hbw + hsub) * 2 + (g == it.first ? 1 : 0)) * kKvRowTile + n;
        const float2 ml = __ldcg(a.part_ml + part);
        alignas(16) float y[V];
        if constexpr (V >= 4) {
#pragma unroll
          for (int j = 0; j < V / 4; ++j)
            *reinterpret_cast<float4*>(y + 4 * j) = __ldcg(reinterpret_cast<const float4*>(a.part_o + part * D + j * 128) + lane);
        } else {
          *reinterpret_cast<float2*>(y) = __ldcg(reinterpret_cast<const float2*>(a.part_o + part * D) + lane);
        }
        const float mn = fmaxf(m, ml.x);
        if (mn > -INFINITY) {
          const float f = ex2(m - mn), w = ex2(ml.x - mn);
          l = l * f + ml.y * w;
#pragma unroll
          for (int j = 0; j < V; ++j) o[j] = o[j] * f + y[j] * w;
          m = mn;
        }
      }
      __syncthreads();          // the previous item's sums are no longer read
      if constexpr (V >= 4) {
#pragma unroll
        for (int j = 0; j < V / 4; ++j)
          *(reinterpret_cast<float4*>(&s_o[warp][j * 128]) + lane) = *reinterpret_cast<float4*>(o + 4 * j);
      } else {
        *(reinterpret_cast<float2*>(s_o[warp]) + lane) = *reinterpret_cast<float2*>(o);
      }
      if (lane == 0) s_ml[warp] = make_float2(m, l);
      __syncthreads();
      for (int e = 2 * tid; e < dim; e += 2 * kJoinThreads) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, s_ml[w].x);
        float L = 0.f, y0 = 0.f, y1 = 0.f;
        if (M > -INFINITY) {
#pragma unroll
          for (int w = 0; w < kJoinWarps; ++w) {
            const float f = ex2(s_ml[w].x - M);
            L += s_ml[w].y * f;
            y0 += s_o[w][e] * f;
            y1 += s_o[w][e + 1] * f;
          }
        }
        const float inv = L > 0.f ? 1.f / L : 0.f;
        *reinterpret_cast<uint32_t*>(a.out + (int64_t)(q0 + row / group) * a.ldo +
                                     (int64_t)(hk * group + row % group) * dim + e) = Elem<E>::from2(y0 * inv, y1 * inv);
      }
    }
  }
}

template <class E, int D>
cudaError_t launch_decode(const KvAttendArgs& a, int num_sms, cudaStream_t st) {
  const int grid = num_sms * (D <= 128 ? kDecCtas : 2);
  if (a.softcap > 0.f) kv_decode_kernel<E, D, true><<<grid, kDecThreads, 0, st>>>(a);
  else kv_decode_kernel<E, D, false><<<grid, kDecThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(4 * num_sms);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<E, D>, a, (int64_t)grid * kDecWarps / a.hbw);
}

template <class E>
cudaError_t decode_dispatch(const KvAttendArgs& a, int num_sms, cudaStream_t st) {
  if (a.kv.head_dim <= 64) return launch_decode<E, 64>(a, num_sms, st);
  if (a.kv.head_dim <= 128) return launch_decode<E, 128>(a, num_sms, st);
  return launch_decode<E, 256>(a, num_sms, st);
}

}  // namespace

int64_t kv_attend_parts(int num_sms) { return (int64_t)num_sms * kDecCtas * kDecWarps * 2 * kKvRowTile; }
int32_t kv_attend_cols(int32_t head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

cudaError_t launch_kv_decode(const KvAttendArgs& args, int dtype, int num_sms, cudaStream_t st) {
  KvAttendArgs a = args;
  // warps that work on neighbouring heads of the same tokens: the largest of
  // 4, 2, 1 that divides the key heads
  a.hbw = a.kv.heads_kv % 4 == 0 ? 4 : a.kv.heads_kv % 2 == 0 ? 2 : 1;
  return dtype == 0 ? decode_dispatch<__half>(a, num_sms, st) : decode_dispatch<__nv_bfloat16>(a, num_sms, st);
}

}  // namespace slora
