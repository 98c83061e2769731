// slora_kv_attend over a cache held in 4 bits: a warp per (token, query head).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "kv_q4.cuh"

namespace slora {
namespace {

constexpr int kThreads = 256;

template <class E>
__global__ void __launch_bounds__(kThreads) kv_q4_attend_kernel(const __grid_constant__ KvAttendArgs a) {
  __shared__ float s_q[kThreads / 32][kKvMaxHeadDim];
  const KvDev& d = a.kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dim = d.head_dim, ng = d.groups;
  const int group = d.heads_q / d.heads_kv;
  const int64_t plane = (int64_t)d.max_rows * d.max_blocks;
  const float sc = kLog2e * a.scale;
  for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + warp; u < (int64_t)a.T * d.heads_q;
       u += (int64_t)gridDim.x * (kThreads / 32)) {
    const int t = (int)(u / d.heads_q), h = (int)(u - (int64_t)t * d.heads_q), hk = h / group;
    const int req = d.tok_req[t], pos = d.tok_pos[t];
    if (req < 0) continue;
    const int row = dbg_index(d.req[req].w, d.max_rows, d.error);
    const int32_t* tab = d.table + 2 * a.layer * plane + (int64_t)row * d.max_blocks;
    __syncwarp();
    for (int e = lane; e < dim; e += 32) s_q[warp][e] = Elem<E>::to(a.q[t * a.ldq + h * dim + e]);
    for (int e = dim + lane; e < 32 * ng; e += 32) s_q[warp][e] = 0.f;
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[kKvMaxHeadDim / 32] = {};
    for (int j0 = 0; j0 <= pos; j0 += 32) {
      const int j = j0 + lane;
      const uint8_t *kr = nullptr, *vr = nullptr;
      if (j <= pos) {
        const int b = (int)a.per_page_div.div((uint32_t)j), off = j - b * d.per_page;
        const int kp = tab[b], vp = tab[plane + b];
        if ((uint32_t)kp < (uint32_t)d.num_pages && (uint32_t)vp < (uint32_t)d.num_pages) {
          kr = reinterpret_cast<const uint8_t*>(d.pool) + q4_row(d, kp, off);
          vr = reinterpret_cast<const uint8_t*>(d.pool) + q4_row(d, vp, off);
        } else {
          report_err(d.error, kErrInvalid);
        }
      }
      float s = -INFINITY;
      if (kr) {
        s = 0.f;
        const uint32_t* codes = reinterpret_cast<const uint32_t*>(kr + hk * 16 * ng);
        const uint16_t* Ms = reinterpret_cast<const uint16_t*>(kr + d.heads_kv * 16 * ng) + hk * ng;
        for (int g = 0; g < ng; ++g) {
          float x = 0.f;
          for (int k4 = 0; k4 < 4; ++k4) {
            const uint32_t c = codes[k4 * ng + g];
            for (int e = 0; e < 8; ++e)
              x += (float)((int)(c >> (16 * (e & 1) + 4 * (e >> 1)) & 15) - 7) * s_q[warp][32 * g + 8 * k4 + e];
          }
          s += x * (Elem<E>::to(Ms[g]) * 0.125f);
        }
        s = a.softcap > 0.f ? capped<true>(s, sc, a.cap_t, a.cap2) : s * sc;
      }
      float mn = s;
      for (int x = 16; x; x >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, x));
      mn = fmaxf(mn, m);
      const float f = mn == m ? 1.f : ex2(m - mn);
      m = mn;
      const float p = ex2(s - (m == -INFINITY ? 0.f : m));
      l = l * f + p;
      for (int g = 0; g < ng; ++g) o[g] *= f;
      for (int i = 0; i < min(32, pos + 1 - j0); ++i) {
        const uint8_t* v = reinterpret_cast<const uint8_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vr), i));
        const float pi = __shfl_sync(0xffffffffu, p, i);
        if (!v) continue;
        const uint16_t* codes = reinterpret_cast<const uint16_t*>(v + hk * 16 * ng);
        const uint16_t* Ms = reinterpret_cast<const uint16_t*>(v + d.heads_kv * 16 * ng) + hk * ng;
        for (int g = 0; g < ng; ++g)
          o[g] += pi * q4_value(codes[(lane >> 2) * ng + g] >> (4 * (lane & 3)) & 15, Elem<E>::to(Ms[g]));
      }
    }
    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int g = 0; g < ng; ++g) {
      const int e = 32 * g + lane;
      if (e < dim) a.out[t * a.ldo + h * dim + e] = (uint16_t)Elem<E>::from2(o[g] * inv, 0.f);
    }
  }
}

}  // namespace

cudaError_t launch_kv_q4_decode(const KvAttendArgs& a, int dtype, int num_sms, bool, cudaStream_t st) {
  auto kernel = dtype == 0 ? kv_q4_attend_kernel<__half> : kv_q4_attend_kernel<__nv_bfloat16>;
  kernel<<<8 * num_sms, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace slora
