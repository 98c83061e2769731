// The 4-bit form of cached keys and values (slora_kv_q4_create), shared by the
// kernels that write and read it.
//
// 32 elements of a head are a group; ng = ceil(head_dim / 32) of them a head, the
// last one filled up with zeros.  With m the group's element of largest magnitude
// and M = |m| rounded up to five significant bits, with m's sign,
//     k = clamp(floor(8 x / M + 1/2), -7, 8)   stands for   M k / 8.
// k has at most three significant bits where it is odd, so M k / 8 has at most
// eight: a number of both 16-bit types, and every kernel reads the same one.
// Groups with an element that is not finite have M = NaN.
//
// A token's row: 16 ng bytes of codes c = k + 7 a head, head by head, then M [head]
// [group] in the storage type.  The codes of element e = 32 g + r of a head lie where
// the attention's kernels want them, so that one lane's share of all groups is one
// load:
//   K  word (r / 8) ng + g of the head, bits 16 (r % 2) + 4 (r % 8 / 2): the four lanes
//      of a matrix row hold 8 elements of every group each, in pairs 16 bits apart;
//   V  16 bits number (r / 4) ng + g, bits 4 (r % 4): the eight lanes of a matrix
//      column hold 4 elements of every group each.
#pragma once

#include "kv.cuh"
#include "kv.h"

namespace slora {

constexpr int kQ4Group = 32;

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float y;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// |M| of a group whose largest magnitude is a: five significant bits, at least the
// unit below which the storage type's products would lose bits, at most the largest
// such number (finite values past it are held as it); NaN unless a is finite.
template <class E>
__device__ __forceinline__ float q4_scale(float a) {
  constexpr float kFinest = Elem<E>::kBf16 ? 0x1p-100f : 0x1p-21f, kPerFinest = Elem<E>::kBf16 ? 0x1p100f : 0x1p21f;
  constexpr float kLargest = Elem<E>::kBf16 ? 31.f * 0x1p123f : 31.f * 0x1p11f;
  if (!(a <= 3.402823466e38f)) return __uint_as_float(0x7fffffffu);
  const float up = __uint_as_float((__float_as_uint(a) + 0x7ffffu) & 0xfff80000u);
  return fminf(a < 16.f * kFinest ? ceilf(a * kPerFinest) * kFinest : up, kLargest);
}
// What a code stands for.
__device__ __forceinline__ float q4_value(uint32_t code, float M) { return (float)((int)code - 7) * (M * 0.125f); }

// Where a token's row begins; page and token of the page from a slot page * P + t % P.
__device__ __forceinline__ int64_t q4_row(const KvDev& d, int page, int in_page) {
  return page * d.page_bytes + (int64_t)in_page * d.row_bytes;
}

}  // namespace slora
