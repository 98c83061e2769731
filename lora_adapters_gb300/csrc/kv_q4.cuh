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
template <class E>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t y;
  if constexpr (Elem<E>::kBf16) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  else asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
template <class E>
__device__ __forceinline__ uint32_t fma2x16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t y;
  if constexpr (Elem<E>::kBf16) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
  else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
  return y;
}
// Codes become numbers in two steps, both exact: k / 8 = (c - 7) / 8 (from 1024 + c, or
// 128 + c in bf16, which is the code with an exponent's bits around it), then k / 8 M.
// The codes in bits 0-3, 4-7, 8-11 and 12-15 of both halves of w, as pairs of numbers; M twice.
template <class E>
__device__ __forceinline__ void q4_pairs(uint32_t w, uint32_t M, uint32_t (&y)[4]) {
  if constexpr (Elem<E>::kBf16) {
    constexpr uint32_t kBase = 0x43004300u, kEighth = 0x3e003e00u, kOff = 0xc187c187u;    // 128, 1 / 8, -135 / 8
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mul2<E>(fma2x16<E>((w >> 4 * i & 0x000f000fu) | kBase, kEighth, kOff), M);
  } else {
    constexpr uint32_t kBase = 0x64006400u, kEighth = 0x30003000u, kOff = 0xd807d807u;    // 1024, 1 / 8, -1031 / 8
    constexpr uint32_t kEighth16 = 0x20002000u, kOff16 = 0xc870c870u;                     // 1 / 128, -71 / 8
    const uint32_t h = w >> 8;
    y[0] = mul2<E>(fma2x16<E>((w & 0x000f000fu) | kBase, kEighth, kOff), M);
    y[1] = mul2<E>(fma2x16<E>((w & 0x00f000f0u) | kBase, kEighth16, kOff16), M);
    y[2] = mul2<E>(fma2x16<E>((h & 0x000f000fu) | kBase, kEighth, kOff), M);
    y[3] = mul2<E>(fma2x16<E>((h & 0x00f000f0u) | kBase, kEighth16, kOff16), M);
  }
}
// A lane's share of a head: the words that hold 8 elements of every group (c: the
// quarter's first byte), and the scales of the groups (m).
template <int NG>
__device__ __forceinline__ void q4_load(const uint8_t* c, const uint8_t* m, uint32_t (&w)[NG], uint32_t (&s)[(NG + 1) / 2]) {
  if constexpr (NG % 4 == 0) {
#pragma unroll
    for (int g = 0; g < NG; g += 4) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(c) + g / 4);
      w[g] = x.x; w[g + 1] = x.y; w[g + 2] = x.z; w[g + 3] = x.w;
      const uint2 y = __ldg(reinterpret_cast<const uint2*>(m) + g / 4);
      s[g / 2] = y.x; s[g / 2 + 1] = y.y;
    }
  } else if constexpr (NG == 2) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(c));
    w[0] = x.x; w[1] = x.y;
    s[0] = __ldg(reinterpret_cast<const uint32_t*>(m));
  } else {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      w[g] = __ldg(reinterpret_cast<const uint32_t*>(c) + g);
      const uint32_t h = __ldg(reinterpret_cast<const uint16_t*>(m) + g);
      s[g / 2] = g & 1 ? s[g / 2] | h << 16 : h;
    }
  }
}
// The 8 consecutive elements of group g in such a share as pairs of numbers: of a key in
// their order; of a value (0, 4), (1, 5), (2, 6), (3, 7).
template <class E, int NG>
__device__ __forceinline__ void q4_eight(const uint32_t (&w)[NG], const uint32_t (&m)[(NG + 1) / 2], int g, bool value,
                                         uint32_t (&y)[4]) {
  const uint32_t M = __byte_perm(m[g / 2], 0, g & 1 ? 0x3232 : 0x1010);
  // (a value's codes: the share's 16-bit words number g, elements 0-3, and NG + g, 4-7)
  const uint32_t sel = (g & 1 ? 0x32 : 0x10) | ((NG + g) & 1 ? 0x7600 : 0x5400);
  q4_pairs<E>(value ? __byte_perm(w[g / 2], w[(NG + g) / 2], sel) : w[g], M, y);
}
// Such pairs of a value in the order of the elements.
__device__ __forceinline__ uint4 q4_in_order(const uint32_t (&y)[4]) {
  return make_uint4(__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410), __byte_perm(y[0], y[1], 0x7632),
                    __byte_perm(y[2], y[3], 0x7632));
}

// Where a token's row begins: token `in_page` of a page.
__device__ __forceinline__ int64_t q4_row(const KvDev& d, int page, int in_page) {
  return page * d.page_bytes + (int64_t)in_page * d.row_bytes;
}

}  // namespace slora
