// slora_kv_plan and slora_kv_append: block tables and slot maps from request
// lengths, and the norm, rotation and store of a step's queries, keys and
// values (include/slora.h).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kv.cuh"
#include "kv.h"

namespace slora {
namespace {

// ================================================================ plan
// Per request r, with len = ctx + new:
//   q_start_r = sum of the earlier requests' new tokens,
//   first_r   = ceil(ctx / P), opened_r = ceil(len / P) - first_r,
//   open_r    = sum of the earlier requests' opened blocks;
// block first_r + i of row_r gets pages[open_r + i], and token t of request r
// at position p = ctx + t - q_start_r sits in slot page(p / P) * P + p % P.
//
// One launch.  Every CTA computes the two prefix sums over all requests for
// itself (R <= 4096: a few loads and one block scan, cheaper than a second
// launch or a grid-wide wait), then takes tiles of 8 or 32 tokens.  A tile's
// pages go through shared memory, because `pages` is contiguous along
// (layer, K/V) and the slot map along tokens.  A fresh block's table entries
// are written by the token at its first position, which is always a new one.
constexpr int kPlanThreads = 512;
constexpr int kPlanTokens = 32;      // tokens of a tile at most
constexpr int kPlanTokensFew = 8;    // for few tokens: more CTAs, one load a thread
constexpr int kPlanPlanes = 64;      // (layer, K/V) planes per pass

constexpr int kPlanSums = 4;
struct PlanSmem {
  int32_t q_start[kKvMaxRequests + 1];
  int32_t open[kKvMaxRequests + 1];    // first block of each request in `pages`
  int32_t warp_sum[kPlanSums][kPlanThreads / 32];
  int32_t page[kPlanTokens][kPlanPlanes + 1];
  int32_t t_row[kPlanTokens], t_block[kPlanTokens], t_open[kPlanTokens], t_off[kPlanTokens];
};

// Sums stay below 2^31: what is larger is larger than T or n_blocks anyway.
__device__ __forceinline__ int32_t sat_add(int32_t a, int32_t b) {
  return (int32_t)min((uint32_t)a + (uint32_t)b, 0x7fffffffu);
}

// The attention's work for one request: decode units (row tiles of its (token,
// head of the group) rows times 16-token units of its length) or, for a chunk,
// 128-key tiles of every pair of row tiles, up to the pair's last position, and
// the pair's own cost.
__device__ __forceinline__ void plan_work(const KvPlanArgs& a, int fresh, int ctx, int32_t* dec, int32_t* tc) {
  const int64_t rows = (int64_t)fresh * (a.kv.heads_q / a.kv.heads_kv);
  const int len = ctx + fresh;
  *dec = *tc = 0;
  if (a.tpt > 0 && rows > kKvChunkRows) {
    // pairs of S = 2 tpt tokens; full pair i needs floor((ctx + S + 127 + S i) / 128)
    // key tiles.  S is even, so 64 pairs on it is S / 2 tiles more: one step for all the
    // pairs with the same i % 64, whatever the lengths
    const int step = 2 * a.tpt, full = fresh / step, first = ctx + step + kKvTile - 1;
    int64_t n = (int64_t)kKvPairUnits * full;
    for (int i = 0; i < min(full, 64); ++i) {
      const int64_t same = (full - i + 63) / 64;
      n += same * ((first + step * i) / kKvTile) + same * (same - 1) / 2 * a.tpt;
    }
    if (fresh % step) n += kKvPairUnits + (len + kKvTile - 1) / kKvTile;
    *tc = (int32_t)min(n, (int64_t)0x7fffffff);
  } else {
    *dec = (int32_t)min((rows + kKvRowTile - 1) / kKvRowTile * (((int64_t)len + kKvUnit - 1) / kKvUnit), (int64_t)0x7fffffff);
  }
}

__device__ __forceinline__ int32_t ceil_pages(const KvPlanArgs& a, int32_t tokens) {   // tokens <= 2^30
  return (int32_t)a.per_page_div.div((uint32_t)(tokens + a.kv.per_page - 1));
}
struct PlanReq {
  int32_t row, ctx, fresh;   // row -1: left out
  int32_t opened;            // blocks the step opens
};
__device__ __forceinline__ PlanReq plan_req(const KvPlanArgs& a, int r) {
  PlanReq q;
  q.row = a.row ? __ldg(a.row + r) : r;
  q.ctx = __ldg(a.ctx + r);
  q.fresh = __ldg(a.fresh + r);
  q.opened = 0;
  const int64_t room = (int64_t)a.kv.max_blocks * a.kv.per_page;
  if (q.row < 0 || q.row >= a.kv.max_rows || q.ctx < 0 || q.fresh < 0 || q.fresh > a.max_new ||
      (int64_t)q.ctx + q.fresh > room)
    q.row = -1;
  else
    q.opened = ceil_pages(a, q.ctx + q.fresh) - ceil_pages(a, q.ctx);
  return q;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const __grid_constant__ KvPlanArgs a) {
  extern __shared__ int32_t plan_smem[];
  PlanSmem& sm = *reinterpret_cast<PlanSmem*>(plan_smem);
  const KvDev& d = a.kv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = d.per_page;
  // ---- prefix sums over the requests, each thread a run of `per` of them:
  // new tokens, opened blocks and (the first CTA alone) the attention's work
  const int per = (a.R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
  const bool lead = blockIdx.x == 0;
  int32_t own[kPlanSums] = {}, inc[kPlanSums] = {}, at[kPlanSums] = {}, tot[kPlanSums] = {};
  bool bad = false;
  for (int r = r0; r < r1; ++r) {
    const PlanReq q = plan_req(a, r);
    if (q.row < 0) {
      bad = true;
      continue;
    }
    own[0] = sat_add(own[0], q.fresh);
    own[1] = sat_add(own[1], q.opened);
    if (lead) {
      int32_t dec, tc;
      plan_work(a, q.fresh, q.ctx, &dec, &tc);
      own[2] = sat_add(own[2], dec);
      own[3] = sat_add(own[3], tc);
    }
  }
#pragma unroll
  for (int k = 0; k < kPlanSums; ++k) {
    if (k >= 2 && !lead) break;
    inc[k] = own[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t v = __shfl_up_sync(0xffffffffu, inc[k], o);
      if (lane >= o) inc[k] = sat_add(inc[k], v);
    }
    if (lane == 31) sm.warp_sum[k][warp] = inc[k];
  }
  __syncthreads();
  const int busy = min(kPlanThreads / 32, (a.R + 32 * max(per, 1) - 1) / (32 * max(per, 1)));   // warps with requests
#pragma unroll
  for (int k = 0; k < kPlanSums; ++k) {
    if (k >= 2 && !lead) break;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w >= busy && w > warp) break;
      if (w == warp) at[k] = tot[k];
      tot[k] = sat_add(tot[k], sm.warp_sum[k][w]);
    }
    const int32_t before = __shfl_up_sync(0xffffffffu, inc[k], 1);
    if (lane) at[k] = sat_add(at[k], before);
  }
  // more tokens than T or more blocks than pages: nobody has a place that can
  // be relied on, every request is left out
  const bool none = tot[0] > a.T || tot[1] > a.n_blocks;
  // more work than 31 bits count: no attention
  const bool idle = none || tot[2] == 0x7fffffff || tot[3] == 0x7fffffff;
  if (none) at[0] = at[1] = tot[0] = 0;
  if (idle) at[2] = at[3] = tot[2] = tot[3] = 0;
  if ((bad || idle) && lead) report_err(d.error, kErrInvalid);
  const int32_t tot_t = tot[0];
  for (int r = r0; r < r1; ++r) {
    const PlanReq q = plan_req(a, r);
    const bool in = q.row >= 0 && !none;
    sm.q_start[r] = at[0];
    sm.open[r] = at[1];
    if (lead) {
      d.q_start[r] = at[0];
      d.dec_off[r] = at[2];
      d.tc_off[r] = at[3];
      d.kv_len[r] = in ? q.ctx + q.fresh : 0;
      d.req[r] = in ? make_int4(at[0], q.fresh, q.ctx + q.fresh, q.row) : make_int4(at[0], 0, 0, 0);
      if (in && !idle) {
        int32_t dec, tc;
        plan_work(a, q.fresh, q.ctx, &dec, &tc);
        at[2] += dec;
        at[3] += tc;
      }
    }
    if (in) {
      at[0] += q.fresh;
      at[1] += q.opened;
    }
  }
  if (tid == 0) {
    sm.q_start[a.R] = tot_t;
    if (lead) {
      d.q_start[a.R] = tot_t;
      d.dec_off[a.R] = tot[2];
      d.tc_off[a.R] = tot[3];
    }
  }
  __syncthreads();
  // ---- tokens
  const int planes = 2 * d.layers, tile = a.tile;
  for (int t0 = blockIdx.x * tile; t0 < a.T; t0 += gridDim.x * tile) {
    if (tid < tile) {
      const int t = t0 + tid;
      int req = -1, pos = -1, row = -1, block = 0, open = -1;
      if (t < tot_t) {
        int lo = 0, hi = a.R - 1;          // the last request that starts at or before t
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (sm.q_start[mid] <= t) lo = mid;
          else hi = mid - 1;
        }
        const PlanReq q = plan_req(a, lo);
        req = lo;
        pos = q.ctx + t - sm.q_start[lo];
        row = q.row;
        block = (int)a.per_page_div.div((uint32_t)pos);
        const int first = ceil_pages(a, q.ctx);
        if (block >= first) open = sm.open[lo] + block - first;
      }
      if (t < a.T) {
        d.tok_req[t] = req;
        d.tok_pos[t] = pos;
      }
      sm.t_row[tid] = row;
      sm.t_block[tid] = block;
      sm.t_open[tid] = open;
      sm.t_off[tid] = pos - block * P;
    }
    for (int p0 = 0; p0 < planes; p0 += kPlanPlanes) {
      const int np = min(kPlanPlanes, planes - p0);
      __syncthreads();
#pragma unroll 4
      for (int i = tid; i < tile * kPlanPlanes; i += kPlanThreads) {
        const int t = i / kPlanPlanes, p = i % kPlanPlanes;
        int page = -1;
        if (p < np && sm.t_row[t] >= 0) {
          if (sm.t_open[t] >= 0) {
            page = __ldg(a.pages + (int64_t)sm.t_open[t] * planes + p0 + p);
          } else {   // a block that was there before: not written in this launch
            page = d.table[((int64_t)(p0 + p) * d.max_rows + sm.t_row[t]) * d.max_blocks + sm.t_block[t]];
          }
          if (page < 0 || page >= d.num_pages) {
            report_err(d.error, kErrInvalid);
            page = -1;
          }
        }
        sm.page[t][p] = page;
      }
      __syncthreads();
#pragma unroll 4
      for (int i = tid; i < kPlanPlanes * tile; i += kPlanThreads) {
        const int p = i / tile, t = i % tile;
        if (p >= np || t0 + t >= a.T) continue;
        const int page = sm.page[t][p];
        d.slots[(int64_t)(p0 + p) * d.max_tokens + t0 + t] = page < 0 ? -1 : page * P + sm.t_off[t];
        if (sm.t_open[t] >= 0 && sm.t_off[t] == 0)
          d.table[((int64_t)(p0 + p) * d.max_rows + sm.t_row[t]) * d.max_blocks + sm.t_block[t]] = page;
      }
    }
    __syncthreads();
  }
}

// ================================================================ append
// One head vector x of head_dim elements at a time:
//   x <- x * rsqrt(mean(x^2) + eps) * w            (optional)
//   (a, b) <- m (a cos - b sin, a sin + b cos)     per pair, angle pos * f_i
// in fp32, rounded once.  A head takes G = 8, 16 or 32 lanes (at least
// head_dim / 8), each lane eight consecutive elements (one 16-byte load and
// store); the sum of squares is a shuffle reduction over G lanes, and the half
// layout's partner element sits rot_dim / 16 lanes away.  Values are copied
// bit for bit by the same lanes.
//
// Bound: memory, each element read and written once, as long as an iteration
// (one load and store a lane) stays near a hundred instructions.  So a warp
// takes one token and a share of its heads (all of them when there are tokens
// enough): its lanes' cosines and sines, the same in every head, are worked
// out once and stay in registers, queries, keys and values have loops of their
// own, and nothing waits at a barrier.  kAppendAhead loads a lane are on their
// way before the first is worked on.  Measured: 8256 tokens of 56 heads, normed,
// half of each head turned, 46.6 us (5.0 TB/s); the half layout over whole heads
// 56 us (its exchange takes eight shuffles a lane), not normed 45.6 us (four
// shuffles; 64 bytes of spills at 64 registers); 256 tokens of 96 heads 6.9 us, at
// the cost of the call.
constexpr int kAppendThreads = 256;
constexpr int kAppendAhead = 4;

template <class E, bool NORM, bool INTER, int G>
struct AppendLane {
  static constexpr int kPerWarp = 32 / G;        // heads a warp takes at a time
  int lane, li, partner;                         // lane in the head, the half layout's partner in the warp
  bool live, turned;
  float inv_d, eps;
  float2 cs[INTER ? 4 : 8];

  // Norm and rotation of this lane's eight elements of a head.
  __device__ __forceinline__ uint4 head(uint4 r, const float* w) const {
    float x[8];
    unpack8<E>(r, x);
    if (NORM) {
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        s0 += x[e] * x[e];
        s1 += x[e + 1] * x[e + 1];
      }
      float ss = s0 + s1;
#pragma unroll
      for (int o = G >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float rs = rsqrtf(ss * inv_d + eps);
      const float4 w0 = *reinterpret_cast<const float4*>(w), w1 = *reinterpret_cast<const float4*>(w + 4);
      x[0] *= rs * w0.x; x[1] *= rs * w0.y; x[2] *= rs * w0.z; x[3] *= rs * w0.w;
      x[4] *= rs * w1.x; x[5] *= rs * w1.y; x[6] *= rs * w1.z; x[7] *= rs * w1.w;
    }
    if (INTER) {
      if (turned) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float u = x[2 * e], z = x[2 * e + 1];
          x[2 * e] = u * cs[e].x - z * cs[e].y;
          x[2 * e + 1] = u * cs[e].y + z * cs[e].x;
        }
      }
    } else {
      // the partner's elements: normed by their own lane, or as they were loaded
      float y[8];
      if (NORM) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], partner);
      } else {
        uint4 o;
        o.x = __shfl_sync(0xffffffffu, r.x, partner);
        o.y = __shfl_sync(0xffffffffu, r.y, partner);
        o.z = __shfl_sync(0xffffffffu, r.z, partner);
        o.w = __shfl_sync(0xffffffffu, r.w, partner);
        unpack8<E>(o, y);
      }
      if (turned) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * cs[e].x + y[e] * cs[e].y;
      }
    }
    return pack8<E>(x);
  }
  // Iterations [i0, i1) of kPerWarp heads each, of `heads`; src and dst point
  // to this lane's elements of iteration 0, dst may be NULL.  WORK: norm and
  // rotate, else copy.
  template <bool WORK>
  __device__ __forceinline__ void run(const uint16_t* src, uint16_t* dst, int i0, int i1, int heads, int step,
                                      const float* w) const {
    const int h0 = lane / G;
    for (int ib = i0; ib < i1; ib += kAppendAhead) {
      uint4 raw[kAppendAhead];
#pragma unroll
      for (int j = 0; j < kAppendAhead; ++j)
        raw[j] = live && ib + j < i1 && (ib + j) * kPerWarp + h0 < heads
                     ? *reinterpret_cast<const uint4*>(src + (ib + j) * step)
                     : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < kAppendAhead; ++j) {
        if (ib + j >= i1) break;                 // the same for the whole warp
        const uint4 r = WORK ? head(raw[j], w) : raw[j];
        if (live && dst && (ib + j) * kPerWarp + h0 < heads) *reinterpret_cast<uint4*>(dst + (ib + j) * step) = r;
      }
    }
  }
};

template <class E, bool NORM, bool INTER, int G>
__global__ void __launch_bounds__(kAppendThreads, NORM && !INTER ? 3 : 4) kv_append_kernel(const __grid_constant__ KvAppendArgs a) {
  using Lane = AppendLane<E, NORM, INTER, G>;
  __shared__ __align__(16) float s_w[2][kKvMaxHeadDim];        // norm weights of queries and keys
  const KvDev& d = a.kv;
  const int tid = threadIdx.x;
  const int D = d.head_dim;
  if (NORM) {
    for (int i = tid; i < 2 * D; i += kAppendThreads)
      s_w[i >= D][i >= D ? i - D : i] = Elem<E>::to(i >= D ? a.kw[i - D] : a.qw[i]);
    __syncthreads();
  }
  const int unit = blockIdx.x * (kAppendThreads / 32) + (tid >> 5);     // T * parts < 2^31
  const int t = unit / a.parts, part = unit - t * a.parts;
  if (t >= a.T) return;
  const int pos = d.tok_pos[t];
  const int32_t* slots = d.slots + (int64_t)2 * a.layer * d.max_tokens + t;
  const int64_t pool_rows = (int64_t)d.num_pages * d.per_page;
  int ks = slots[0], vs = slots[d.max_tokens];
  if (ks >= 0) ks = dbg_index(ks, pool_rows, d.error);
  if (vs >= 0) vs = dbg_index(vs, pool_rows, d.error);
  if (pos < 0) return;                           // a token without a request
  Lane ln;
  ln.lane = tid & 31;
  ln.li = ln.lane & (G - 1);
  ln.live = ln.li * 8 < D;
  const int half = a.rot_dim >> 4;               // half layout: lanes between the halves
  const int pl = ln.li < half ? ln.li + half : ln.li - half;
  ln.turned = ln.li < 2 * half;
  ln.partner = (ln.lane & ~(G - 1)) | (ln.turned ? pl : ln.li);
  ln.inv_d = 1.f / (float)D;
  ln.eps = a.eps;
  // Cosine and sine of this lane's pairs: the angle as a fraction of a turn modulo
  // one, a signed 64-bit number that wraps around without error, then in fp32
  // (2^-25 turn); within half a turn the approximate functions are good to 2^-21,
  // 1/1024 of fp16's unit and 2^-13 of bf16's.
#pragma unroll
  for (int j = 0; j < (INTER ? 4 : 8); ++j) {
    const int pi = INTER ? ln.li * 4 + j : (ln.li < half ? ln.li : pl) * 8 + j;
    float ang = 0.f;
    if (ln.turned) ang = (float)(int64_t)((uint64_t)pos * __ldg(a.freq + pi)) * (0x1p-63f * 3.14159265358979f);
    ln.cs[j] = make_float2(__cosf(ang) * a.mscale, __sinf(ang) * a.mscale);
    if (!INTER && ln.li < half) ln.cs[j].y = -ln.cs[j].y;     // lower elements: x cos - y sin, upper: x cos + y sin
  }
  const int nq = (d.heads_q + Lane::kPerWarp - 1) / Lane::kPerWarp, nk = (d.heads_kv + Lane::kPerWarp - 1) / Lane::kPerWarp;
  const int iters = nq + 2 * nk, i0 = iters * part / a.parts, i1 = iters * (part + 1) / a.parts;
  const int at = (ln.lane / G) * D + ln.li * 8, step = Lane::kPerWarp * D;
  const int64_t width = (int64_t)d.heads_kv * D;
  ln.template run<true>(a.q + (int64_t)t * a.ldq + at, a.q_out + (int64_t)t * a.ldqo + at, i0, min(i1, nq), d.heads_q, step,
                        s_w[0] + ln.li * 8);
  ln.template run<true>(a.k + (int64_t)t * a.ldk + at, ks < 0 ? nullptr : d.pool + ks * width + at, max(i0 - nq, 0),
                        min(i1 - nq, nk), d.heads_kv, step, s_w[1] + ln.li * 8);
  ln.template run<false>(a.v + (int64_t)t * a.ldv + at, vs < 0 ? nullptr : d.pool + vs * width + at,
                         max(i0 - nq - nk, 0), i1 - nq - nk, d.heads_kv, step, nullptr);
}

template <class E, bool NORM, bool INTER>
void (*append_kernel(int lanes))(const KvAppendArgs) {
  return lanes == 8 ? kv_append_kernel<E, NORM, INTER, 8> : lanes == 16 ? kv_append_kernel<E, NORM, INTER, 16>
                                                                        : kv_append_kernel<E, NORM, INTER, 32>;
}
template <class E>
void (*append_kernel(bool norm, bool inter, int lanes))(const KvAppendArgs) {
  if (norm) return inter ? append_kernel<E, true, true>(lanes) : append_kernel<E, true, false>(lanes);
  return inter ? append_kernel<E, false, true>(lanes) : append_kernel<E, false, false>(lanes);
}

}  // namespace

cudaError_t prepare_kv_kernels() {
  return cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(PlanSmem));
}

cudaError_t launch_kv_plan(const KvPlanArgs& args, cudaStream_t st) {
  KvPlanArgs a = args;
  // every CTA repeats the sums, so large batches take larger tiles
  a.tile = a.T <= 128 * kPlanTokensFew ? kPlanTokensFew : kPlanTokens;
  const int tiles = std::max(1, (a.T + a.tile - 1) / a.tile);
  kv_plan_kernel<<<std::min(tiles, 1024), kPlanThreads, sizeof(PlanSmem), st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(const KvAppendArgs& args, int dtype, int num_sms, cudaStream_t st) {
  KvAppendArgs a = args;
  const int lanes = a.kv.head_dim <= 64 ? 8 : a.kv.head_dim <= 128 ? 16 : 32, per_warp = 32 / lanes;
  const int iters = (a.kv.heads_q + per_warp - 1) / per_warp + 2 * ((a.kv.heads_kv + per_warp - 1) / per_warp);
  // Few tokens: their heads are shared out over warps, up to 16 warps an SM
  // (256 tokens of 96 heads: 6.9 us with 16, 7.5 with 8, 8.4 with 32).
  a.parts = std::max(1, std::min(iters, 16 * num_sms / a.T));
  const int64_t warps = (int64_t)a.T * a.parts;
  const int grid = (int)((warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
  auto kernel = dtype == 0 ? append_kernel<__half>(a.qw != nullptr, a.interleaved != 0, lanes)
                           : append_kernel<__nv_bfloat16>(a.qw != nullptr, a.interleaved != 0, lanes);
  kernel<<<grid, kAppendThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace slora
