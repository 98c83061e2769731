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

constexpr int kErrInvalid = -1;   // == SLORA_ERR_INVALID

__device__ __forceinline__ void report_err(int32_t* err, int code) {
  if (err) atomicCAS(err, 0, code);
}

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
// launch or a grid-wide wait), then takes tiles of kPlanTokens tokens.  A
// tile's pages go through shared memory, because `pages` is contiguous along
// (layer, K/V) and the slot map along tokens.  A fresh block's table entries
// are written by the token at its first position, which is always a new one.
constexpr int kPlanThreads = 512;
constexpr int kPlanTokens = 32;
constexpr int kPlanPlanes = 64;      // (layer, K/V) planes per pass
constexpr int kPlanPer = kKvMaxRequests / kPlanThreads;   // requests per thread at most

constexpr int kPlanSums = 4;
struct PlanSmem {
  int32_t q_start[kKvMaxRequests + 1];
  int32_t open[kKvMaxRequests + 1];    // first block of each request in `pages`
  int32_t warp_sum[kPlanSums][kPlanThreads / 32];
  int32_t page[kPlanTokens][kPlanPlanes + 1];
  int32_t t_row[kPlanTokens], t_block[kPlanTokens], t_open[kPlanTokens], t_off[kPlanTokens];
  int32_t bad;
};

// Sums stay below 2^31: what is larger is larger than T or n_blocks anyway.
__device__ __forceinline__ int32_t sat_add(int32_t a, int32_t b) {
  return (int32_t)min((uint32_t)a + (uint32_t)b, 0x7fffffffu);
}

// The attention's work for one request: decode units (row tiles of its (token,
// head of the group) rows times 16-token units of its length) or, for a chunk,
// 128-key tiles of every pair of row tiles, up to the pair's last position.
__device__ __forceinline__ void plan_work(const KvPlanArgs& a, int fresh, int ctx, int32_t* dec, int32_t* tc) {
  const int64_t rows = (int64_t)fresh * (a.kv.heads_q / a.kv.heads_kv);
  const int len = ctx + fresh;
  *dec = *tc = 0;
  if (a.tpt > 0 && rows > kKvChunkRows) {
    int32_t n = 0;
    for (int t = 0; t < fresh; t += 2 * a.tpt) n = sat_add(n, (ctx + min(fresh, t + 2 * a.tpt) + kKvTile - 1) / kKvTile);
    *tc = n;
  } else {
    *dec = (int32_t)min((rows + kKvRowTile - 1) / kKvRowTile * (((int64_t)len + kKvUnit - 1) / kKvUnit), (int64_t)0x7fffffff);
  }
}

__device__ __forceinline__ int32_t ceil_pages(int32_t tokens, int32_t P) {
  return tokens / P + (tokens % P != 0);
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
    q.opened = ceil_pages(q.ctx + q.fresh, a.kv.per_page) - ceil_pages(q.ctx, a.kv.per_page);
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
  int32_t own[kPlanSums] = {}, inc[kPlanSums], at[kPlanSums] = {}, tot[kPlanSums] = {};
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
    inc[k] = own[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t v = __shfl_up_sync(0xffffffffu, inc[k], o);
      if (lane >= o) inc[k] = sat_add(inc[k], v);
    }
    if (lane == 31) sm.warp_sum[k][warp] = inc[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPlanSums; ++k) {
    for (int w = 0; w < kPlanThreads / 32; ++w) {
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
      d.row[r] = in ? q.row : 0;
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
  const int planes = 2 * d.layers;
  for (int t0 = blockIdx.x * kPlanTokens; t0 < a.T; t0 += gridDim.x * kPlanTokens) {
    if (tid < kPlanTokens) {
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
        block = pos / P;
        const int first = ceil_pages(q.ctx, P);
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
      for (int i = tid; i < kPlanTokens * kPlanPlanes; i += kPlanThreads) {
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
      for (int i = tid; i < kPlanPlanes * kPlanTokens; i += kPlanThreads) {
        const int p = i / kPlanTokens, t = i % kPlanTokens;
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
// in fp32, rounded once.  A head takes G = 8, 16 or 32 lanes (the power of
// two at or above head_dim / 8), each lane eight consecutive elements (one
// 16-byte load and store); the sum of squares is a shuffle reduction over G
// lanes, and the half layout's partner element sits rot_dim / 16 lanes away.
// Cosines and sines of a token are computed once per CTA and shared by every
// head.  Values are copied bit for bit by the same lanes.
//
// Bound: memory, each element read and written once.
constexpr int kAppendThreads = 256;

struct AppendSmem {
  float2 cs[kKvMaxHeadDim / 2];
  float w[2][kKvMaxHeadDim];
};

template <class E, bool NORM, bool INTER>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ KvAppendArgs a) {
  __shared__ AppendSmem sm;
  const KvDev& d = a.kv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int D = d.head_dim, vecs = D >> 3, half = a.rot_dim >> 1;
  int G = 2;
  while (G < vecs) G <<= 1;
  const int li = lane & (G - 1), per_warp = 32 / G;
  const int heads = d.heads_q + 2 * d.heads_kv;
  const bool live = li < vecs;
  const int64_t width = (int64_t)d.heads_kv * D;
  if (NORM)
    for (int i = tid; i < 2 * D; i += kAppendThreads)
      sm.w[i >= D][i >= D ? i - D : i] = Elem<E>::to(i >= D ? a.kw[i - D] : a.qw[i]);
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int pos = d.tok_pos[t];
    if (pos < 0) continue;     // the same for the whole CTA
    const int32_t* slots = d.slots + (int64_t)2 * a.layer * d.max_tokens + t;
    const int ks = slots[0], vs = slots[d.max_tokens];
    __syncthreads();           // the previous token's cosines are no longer read
    for (int i = tid; i < half; i += kAppendThreads) {
      // the fraction of a turn, exact modulo one turn, as a signed 64-bit number
      const int64_t frac = (int64_t)((uint64_t)pos * a.freq[i]);
      float s, c;
      sincospif((float)frac * 0x1p-63f, &s, &c);
      sm.cs[i] = make_float2(c * a.mscale, s * a.mscale);
    }
    __syncthreads();
    for (int h = (blockIdx.y * (kAppendThreads / 32) + warp) * per_warp + lane / G; h < (heads + per_warp - 1) / per_warp * per_warp;
         h += gridDim.y * (kAppendThreads / 32) * per_warp) {
      const bool is_q = h < d.heads_q, is_k = !is_q && h < d.heads_q + d.heads_kv;
      const uint16_t* src = nullptr;
      uint16_t* dst = nullptr;
      if (is_q) {
        src = a.q + (int64_t)t * a.ldq + (int64_t)h * D;
        dst = a.q_out + (int64_t)t * a.ldqo + (int64_t)h * D;
      } else if (is_k) {
        const int hk = h - d.heads_q;
        src = a.k + (int64_t)t * a.ldk + (int64_t)hk * D;
        if (ks >= 0) dst = d.pool + ks * width + (int64_t)hk * D;
      } else if (h < heads) {
        const int hv = h - d.heads_q - d.heads_kv;
        src = a.v + (int64_t)t * a.ldv + (int64_t)hv * D;
        if (vs >= 0) dst = d.pool + vs * width + (int64_t)hv * D;
      }
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (live && src) raw = *reinterpret_cast<const uint4*>(src + li * 8);
      float x[8];
      unpack8<E>(raw, x);
      float rs = 1.f;
      if (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
        for (int o = G >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = rsqrtf(ss / (float)D + a.eps);
      }
      const float* w = sm.w[is_q ? 0 : 1];
      uint4 oth = make_uint4(0, 0, 0, 0);
      const int step = a.rot_dim >> 4;           // lanes between the halves
      if (!INTER) {                              // every lane takes part in the exchange
        const int from = (lane & ~(G - 1)) | (li < step ? li + step : li < 2 * step ? li - step : li);
        oth.x = __shfl_sync(0xffffffffu, raw.x, from);
        oth.y = __shfl_sync(0xffffffffu, raw.y, from);
        oth.z = __shfl_sync(0xffffffffu, raw.z, from);
        oth.w = __shfl_sync(0xffffffffu, raw.w, from);
      }
      if (is_q || is_k) {
        if (live) {
          if (NORM) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= rs * w[li * 8 + j];
          }
          if (INTER) {
            if (li < 2 * step) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 cs = sm.cs[li * 4 + j];
                const float u = x[2 * j], v = x[2 * j + 1];
                x[2 * j] = u * cs.x - v * cs.y;
                x[2 * j + 1] = u * cs.y + v * cs.x;
              }
            }
          } else if (li < 2 * step) {
            const bool lower = li < step;
            const int pl = lower ? li + step : li - step, pi = (lower ? li : pl) * 8;
            float y[8];
            unpack8<E>(oth, y);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (NORM) y[j] *= rs * w[pl * 8 + j];
              const float2 cs = sm.cs[pi + j];
              x[j] = lower ? x[j] * cs.x - y[j] * cs.y : y[j] * cs.y + x[j] * cs.x;
            }
          }
          raw = pack8<E>(x);
        }
      }
      if (live && dst) *reinterpret_cast<uint4*>(dst + li * 8) = raw;
    }
  }
}

template <class E>
cudaError_t append_dispatch(const KvAppendArgs& a, dim3 grid, cudaStream_t st) {
  if (a.qw) {
    if (a.interleaved) kv_append_kernel<E, true, true><<<grid, kAppendThreads, 0, st>>>(a);
    else kv_append_kernel<E, true, false><<<grid, kAppendThreads, 0, st>>>(a);
  } else {
    if (a.interleaved) kv_append_kernel<E, false, true><<<grid, kAppendThreads, 0, st>>>(a);
    else kv_append_kernel<E, false, false><<<grid, kAppendThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_kv_kernels() {
  return cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(PlanSmem));
}

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t st) {
  const int tiles = std::max(1, (a.T + kPlanTokens - 1) / kPlanTokens);
  kv_plan_kernel<<<std::min(tiles, 1024), kPlanThreads, sizeof(PlanSmem), st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(const KvAppendArgs& a, int dtype, int num_sms, cudaStream_t st) {
  // few tokens: their heads are spread over several CTAs each
  const int warps = kAppendThreads / 32;
  const int heads = a.kv.heads_q + 2 * a.kv.heads_kv;
  int parts = std::max(1, std::min((heads + warps - 1) / warps, 2 * num_sms / std::max(a.T, 1)));
  const dim3 grid(std::min(a.T, 16 * num_sms), parts);
  return dtype == 0 ? append_dispatch<__half>(a, grid, st) : append_dispatch<__nv_bfloat16>(a, grid, st);
}

}  // namespace slora
