// Element conversions, scores and error reports shared by the key-value cache
// kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "internal.h"

namespace slora {

template <class T>
struct Elem;
template <>
struct Elem<__half> {
  static constexpr bool kBf16 = false;
  static __device__ __forceinline__ float to(uint16_t u) { return __half2float(__ushort_as_half(u)); }
  // a pair packed in 32 bits, the first value in the low half
  static __device__ __forceinline__ uint32_t from2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 to2(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  static __device__ __forceinline__ float to(uint16_t u) { return __bfloat162float(__ushort_as_bfloat16(u)); }
  static __device__ __forceinline__ uint32_t from2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 to2(uint32_t u) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
  }
};

template <class E>
__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const float2 a = Elem<E>::to2(r.x), b = Elem<E>::to2(r.y), c = Elem<E>::to2(r.z), e = Elem<E>::to2(r.w);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  x[4] = c.x; x[5] = c.y; x[6] = e.x; x[7] = e.y;
}
template <class E>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(Elem<E>::from2(x[0], x[1]), Elem<E>::from2(x[2], x[3]), Elem<E>::from2(x[4], x[5]),
                    Elem<E>::from2(x[6], x[7]));
}

constexpr int kErrInvalid = -1;   // == SLORA_ERR_INVALID
__device__ __forceinline__ void report_err(int32_t* err, int code) {
  if (err) atomicCAS(err, 0, code);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;
// A capped score in powers of two, log2(e) softcap tanh(t), t = x scale / softcap
// for the product x = q . k; unit = log2(e) scale, cap2 = log2(e) softcap.
//   |t| >= 1/4:  1 - 2 / (1 + e^(2t)), absolute error 2^-22, relative 2^-19.6 at 1/4;
//   below, where that difference cancels:  t (1 - t^2/3 + 2 t^4/15 - 17 t^6/315
//   + 62 t^8/2835), the series of tanh, whose next term is below 2^-26 there.  In
//   it log2(e) softcap t is x unit, so a softcap far above the scores leaves them
//   as they are.
// ANY = false leaves the second out, for softcap up to kCapNear: the error of a
// score is then softcap 2^-22, at most 2^-16, for scores of every size.
constexpr float kCapNear = 64.f;
template <bool ANY>
__device__ __forceinline__ float capped(float x, float unit, float cap_t, float cap2) {
  const float far = fmaf(-2.f * cap2, __fdividef(1.f, 1.f + ex2(x * (2.f * kLog2e * cap_t))), cap2);
  if (!ANY) return far;
  const float t = x * cap_t, u = t * t;
  float p = fmaf(u, 62.f / 2835.f, -17.f / 315.f);
  p = fmaf(u, p, 2.f / 15.f);
  p = fmaf(u, p, -1.f / 3.f);
  const float y = x * unit;
  return fabsf(t) < 0.25f ? fmaf(y * u, p, y) : far;
}

}  // namespace slora
