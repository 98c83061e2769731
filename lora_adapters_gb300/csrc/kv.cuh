// Element conversions shared by the key-value cache kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

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

}  // namespace slora
