// A lane's share of slora_kv_append: norm and rotation of a head's elements in
// registers (kv.cu: 16-bit caches, kv_q4.cu: caches in 4 bits).
#pragma once

#include "kv.cuh"

namespace slora {

constexpr int kAppendAhead = 4;

template <class E, bool NORM, bool INTER, int G>
struct AppendLane {
  static constexpr int kPerWarp = 32 / G;        // heads a warp takes at a time
  int lane, li, partner;                         // lane in the head, the half layout's partner in the warp
  bool live, turned;
  float inv_d, eps;
  float2 cs[INTER ? 4 : 8];

  // Norm and rotation of this lane's eight elements of a head, in fp32.
  __device__ __forceinline__ void turn(uint4 r, const float* w, float (&x)[8]) const {
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
  }
  __device__ __forceinline__ uint4 head(uint4 r, const float* w) const {
    float x[8];
    turn(r, w, x);
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

}  // namespace slora
