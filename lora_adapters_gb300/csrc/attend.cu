// slora_kv_attend: causal attention of a step's tokens over their requests'
// paged keys and values (include/slora.h).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "kv.cuh"
#include "kv.h"

namespace slora {
namespace {

// One warp per (token, query head): the softmax's running maximum m, sum l and
// unnormalised output o over the keys j = 0 .. pos,
//   m' = max(m, s_j);  l <- l e^(m - m') + e^(s_j - m');  o <- o e^(m - m') + e^(s_j - m') v_j.
constexpr int kAttendThreads = 256;

template <class E>
__global__ void __launch_bounds__(kAttendThreads) kv_attend_kernel(const __grid_constant__ KvAttendArgs a) {
  const KvDev& d = a.kv;
  const int lane = threadIdx.x & 31;
  const int D = d.head_dim, P = d.per_page;
  const int group = d.heads_q / d.heads_kv;
  const int64_t width = (int64_t)d.heads_kv * D;
  const int64_t units = (int64_t)a.T * d.heads_q;
  const int64_t plane = (int64_t)d.max_rows * d.max_blocks;
  for (int64_t u = (int64_t)blockIdx.x * (kAttendThreads / 32) + (threadIdx.x >> 5); u < units;
       u += (int64_t)gridDim.x * (kAttendThreads / 32)) {
    const int t = (int)(u / d.heads_q), h = (int)(u - (int64_t)t * d.heads_q);
    const int req = d.tok_req[t];
    if (req < 0) continue;
    const int pos = d.tok_pos[t];
    const int32_t* kt = d.table + 2 * a.layer * plane + (int64_t)d.row[req] * d.max_blocks;
    const int32_t* vt = kt + plane;
    float q[8], o[8], m = -INFINITY, l = 0.f;
    const bool live = lane * 8 < D;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (live) raw = *reinterpret_cast<const uint4*>(a.q + (int64_t)t * a.ldq + (int64_t)h * D + lane * 8);
    unpack8<E>(raw, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = 0.f;
    const uint16_t* base = d.pool + (int64_t)(h / group) * D + lane * 8;
    for (int j = 0; j <= pos; ++j) {
      const int b = j / P, off = j - b * P;
      const int kp = kt[b], vp = vt[b];
      if ((uint32_t)kp >= (uint32_t)d.num_pages || (uint32_t)vp >= (uint32_t)d.num_pages) continue;
      uint4 kr = make_uint4(0, 0, 0, 0), vr = kr;
      if (live) {
        kr = *reinterpret_cast<const uint4*>(base + ((int64_t)kp * P + off) * width);
        vr = *reinterpret_cast<const uint4*>(base + ((int64_t)vp * P + off) * width);
      }
      float k[8], v[8], s = 0.f;
      unpack8<E>(kr, k);
      unpack8<E>(vr, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += q[i] * k[i];
#pragma unroll
      for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= a.scale;
      if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
      const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn);
      m = mn;
      l = l * f + p;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = o[i] * f + p * v[i];
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= inv;
    if (live) *reinterpret_cast<uint4*>(a.out + (int64_t)t * a.ldo + (int64_t)h * D + lane * 8) = pack8<E>(o);
  }
}

}  // namespace

cudaError_t launch_kv_attend(const KvAttendArgs& a, int dtype, int num_sms, cudaStream_t st) {
  const int64_t units = (int64_t)a.T * a.kv.heads_q;
  const int64_t ctas = std::min<int64_t>((units + kAttendThreads / 32 - 1) / (kAttendThreads / 32), 64 * num_sms);
  if (dtype == 0) kv_attend_kernel<__half><<<(int)ctas, kAttendThreads, 0, st>>>(a);
  else kv_attend_kernel<__nv_bfloat16><<<(int)ctas, kAttendThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace slora
