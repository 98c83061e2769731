// slora_kv_append to a cache held in 4 bits, and slora_kv_read of either cache
// (include/slora.h; the format: kv_q4.cuh).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "append.cuh"
#include "kv_q4.cuh"

namespace slora {
namespace {

// ================================================================ append
// Norm and rotation as in kv.cu, a warp per token and share of its heads, eight
// consecutive elements a lane; a group is four lanes.  Bound: instructions, about 150 a
// lane's eight quantised elements: 8090 tokens of 56 heads, normed, half of each head
// turned, 61 to 63 us (181 MB, 59 % of the issue slots); 256 tokens of 96 heads 12.
//
// Codes are those of the formula in exact arithmetic, not of its fp32 evaluation:
//  - a value that comes straight from 16 bits has at most 11 significant bits, a
//    border (2n + 1) M / 16 at most 9, so the two are equal or at least 2^-11 of the
//    border apart.  t = 8 x / M evaluated with an error below 2^-18 and raised by
//    2^-15 then rounds to the right integer, ties upwards;
//  - a rotated key has an error of at most 2^-20.7 of its pair's larger element (angle
//    2^-23.3, cosine and sine 2^-24 more, mscale's product 2^-24: 2^-22.1 each, times the
//    sum of two elements, at most twice the larger rotated one; a product's and a sum's
//    rounding), a normed one of 2^-19.6 (every element's factor 2^-23, the norm's
//    2^-20.9: nine roundings of the sum of squares, halved, and the root's two units).  Where
//    that could change a code, M's rounding or the choice between the two signs, the warp
//    works the elements in question out again in fp64 (exact_scale, exact_codes).  The bound
//    counts from the largest element of the group and of those with its pairs' other halves
//    (one past fp32's range counts as the largest number: its pair's may be finite).  From the
//    head's largest, one outlier had whole heads worked out again (256 tokens with an infinite
//    element a head 178 us, 16 so; 8090 normed ones with one 1000 times the rest 264, 64 so)
constexpr int kAppendThreads = 256;
constexpr float kErrTurned = 0x1.6p-21f, kErrNormed = 0x1.6p-20f;     // 2^-20.5, 2^-19.5

// What the two need of a lane.
struct Exact {
  const uint64_t* freq;
  int64_t pos;
  float mscale, eps;
  double inv_d;                  // 1 / head_dim
  int half;                      // lanes between the halves of the half layout
};

// Element e of eight packed in r.
template <class E>
__device__ __forceinline__ float element(const uint4& r, int e) {
  const uint32_t w = e & 4 ? (e & 2 ? r.w : r.z) : (e & 2 ? r.y : r.x);
  return Elem<E>::to((uint16_t)(e & 1 ? w >> 16 : w));
}

// Normed and rotated elements in fp64, by a whole warp; r: the lane's raw elements, w: its
// weights.  One element at a time, the same of every lane: the calls below ask for few, and
// what unrolled code costs first is its fetch (256 tokens of 96 heads 29 us, 14 as it is).
template <class E, bool NORM, bool INTER, int G>
struct Turned {
  const Exact& ex;
  const float* w;
  const float* wo;               // the partner's weights
  uint4 r, o;                    // own and partner's raw elements
  double rs = 1.0;
  int li, first_pair;
  bool turned, lower;

  __device__ __forceinline__ Turned(const Exact& x, const uint4& raw, const float* weights) : ex(x), w(weights), r(raw), o(raw) {
    const int lane = threadIdx.x & 31;
    li = lane & (G - 1);
    const int pl = li < ex.half ? li + ex.half : li - ex.half;
    turned = li < 2 * ex.half;
    lower = li < ex.half;
    first_pair = INTER ? li * 4 : (lower ? li : pl) * 8;
    wo = INTER || !turned ? w : w + (pl - li) * 8;
    if (!INTER) {
      const int partner = (lane & ~(G - 1)) | (turned ? pl : li);
      o.x = __shfl_sync(0xffffffffu, r.x, partner);
      o.y = __shfl_sync(0xffffffffu, r.y, partner);
      o.z = __shfl_sync(0xffffffffu, r.z, partner);
      o.w = __shfl_sync(0xffffffffu, r.w, partner);
    }
    if (NORM) {
      // squares of 16-bit numbers are exact in fp32; 1 / sqrt(v) from fp32's 22 bits by two
      // of Newton's steps, y <- y (3 - v y^2) / 2, each of which doubles them
      float v[8];
      unpack8<E>(r, v);
      double s0 = 0.0, s1 = 0.0;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        s0 += (double)(v[e] * v[e]);
        s1 += (double)(v[e + 1] * v[e + 1]);
      }
      double ss = s0 + s1;
#pragma unroll 1
      for (int x2 = G >> 1; x2; x2 >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x2);
      ss = fma(ss, ex.inv_d, (double)ex.eps);
      rs = (double)rsqrtf((float)ss);
#pragma unroll
      for (int i = 0; i < 2; ++i) rs = rs * fma(-0.5 * ss * rs, rs, 1.5);
    }
  }
  __device__ __forceinline__ double operator()(int e) const {
    double x = element<E>(r, e);
    if (NORM) x = x * w[e] * rs;                   // (x w exactly: equal magnitudes stay equal)
    if (!turned) return x;
    const int pe = INTER ? e ^ 1 : e;
    double b = INTER ? element<E>(r, pe) : element<E>(o, pe), c, s;
    if (NORM) b = b * wo[pe] * rs;
    sincospi((double)(int64_t)((uint64_t)ex.pos * ex.freq[first_pair + (INTER ? e / 2 : e)]) * 0x1p-63, &s, &c);
    return (x * c + ((INTER ? (e & 1) == 0 : lower) ? -b : b) * s) * (double)ex.mscale;
  }
};

// M of the lane's group, from those of its elements that may be the largest (a bit each).
template <class E, bool NORM, bool INTER, int G>
__device__ __noinline__ float exact_scale(const Exact ex, uint4 r, const float* w, uint32_t largest) {
  const Turned<E, NORM, INTER, G> x(ex, r, w);
  double hi = 0.0, lo = 0.0;
#pragma unroll 1
  for (uint32_t left = __reduce_or_sync(0xffffffffu, largest); left; left &= left - 1) {
    const int e = __ffs(left) - 1;
    const double v = x(e);
    if (largest >> e & 1) {
      hi = fmax(hi, v);
      lo = fmin(lo, v);
    }
  }
#pragma unroll 1
  for (int y = 1; y < 4; y <<= 1) {
    hi = fmax(hi, __shfl_xor_sync(0xffffffffu, hi, y));
    lo = fmin(lo, __shfl_xor_sync(0xffffffffu, lo, y));
  }
  return copysignf(q4_scale<E>(__double2float_ru(fmax(hi, -lo))), hi >= -lo ? 1.f : -1.f);   // (upwards, as M itself)
}
// The codes (packed as K's) with those replaced that `need` has a bit for.
template <class E, bool NORM, bool INTER, int G>
__device__ __noinline__ uint32_t exact_codes(const Exact ex, uint4 r, const float* w, uint32_t need, float M, uint32_t word) {
  const Turned<E, NORM, INTER, G> x(ex, r, w);
#pragma unroll 1
  for (uint32_t left = __reduce_or_sync(0xffffffffu, need); left; left &= left - 1) {
    const int e = __ffs(left) - 1;
    const double v = x(e);
    if (need >> e & 1) {
      // n <= t < n + 1 as fp32 sees t = 8 x / M; the border between n and n + 1 is
      // (n + 1/2) M / 8, compared exactly
      const float am = fabsf(M), n = M == 0.f ? 0.f : floorf(fminf(fmaxf(8.f * (float)v / M, -8.f), 9.f));
      const double y = M < 0.f ? -8.0 * v : 8.0 * v;
      const int k = min(max((int)n + (M != 0.f && y >= (double)((n + 0.5f) * am)), -7), 8);
      const int at = 16 * (e & 1) + 4 * (e >> 1);
      word = (word & ~(15u << at)) | (uint32_t)(k + 7) << at;
    }
  }
  return word;
}

__device__ __forceinline__ float rcp(float x) {     // to one unit of the last place
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t nibbles(float a, float b, float c, float e) {   // of codes k, the first lowest
  return __float_as_uint(fmaf(fmaf(fmaf(e, 16.f, c), 16.f, b), 16.f, a) + (8388608.f + 0x7777));
}
// The codes k of x (inv = 8 / M, bump: by how much 8 x / M is raised), and in d how far
// they are from it before they are held above -8.
__device__ __forceinline__ void round8(const float (&x)[8], float inv, float bump, float (&k)[8], float (&d)[8]) {
  constexpr float kInt = 12582912.f;               // 1.5 * 2^23: adding it rounds to an integer
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = fmaf(x[e], inv, bump), r = (t + kInt) - kInt;
    d[e] = r - t;
    k[e] = fmaxf(r, -7.f);                         // (above 8 only where M is the type's largest)
  }
}

template <class E, bool NORM, bool INTER, int G>
__global__ void __launch_bounds__(kAppendThreads, 3) kv_q4_append_kernel(const __grid_constant__ KvAppendArgs a) {
  using Lane = AppendLane<E, NORM, INTER, G>;
  __shared__ __align__(16) float s_w[2][kKvMaxHeadDim];        // norm weights of queries and keys
  const KvDev& d = a.kv;
  const int tid = threadIdx.x;
  const int D = d.head_dim;
  if (NORM) {
    // zeros past head_dim: the lanes there have zeros for elements, and where the last group is
    // half full their products with the weights are among its elements
    constexpr int kLanes = 8 * G;
    for (int i = tid; i < 2 * kLanes; i += kAppendThreads) {
      const int e = i % kLanes;
      s_w[i / kLanes][e] = e < D ? Elem<E>::to(i < kLanes ? a.qw[e] : a.kw[e]) : 0.f;
    }
    __syncthreads();
  }
  const int unit = blockIdx.x * (kAppendThreads / 32) + (tid >> 5);     // T * parts < 2^31
  const int t = unit / a.parts, part = unit - t * a.parts;
  if (t >= a.T) return;
  const int pos = d.tok_pos[t];
  const int32_t* slots = d.slots + (int64_t)2 * a.layer * d.max_tokens + t;
  int ks = slots[0], vs = slots[d.max_tokens];
  const int64_t pool_slots = (int64_t)d.num_pages * d.per_page;
  if (ks >= 0) ks = dbg_index(ks, pool_slots, d.error);
  if (vs >= 0) vs = dbg_index(vs, pool_slots, d.error);
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
  // one (kv.cu), in fp32 to 2^-25 turn, the functions to 2^-23
#pragma unroll
  for (int j = 0; j < (INTER ? 4 : 8); ++j) {
    const int pi = INTER ? ln.li * 4 + j : (ln.li < half ? ln.li : pl) * 8 + j;
    float ang = 0.f, s, c;
    if (ln.turned) ang = (float)(int64_t)((uint64_t)pos * __ldg(a.freq + pi)) * 0x1p-63f;
    sincospif(ang, &s, &c);
    ln.cs[j] = make_float2(c * a.mscale, s * a.mscale);
    if (!INTER && ln.li < half) ln.cs[j].y = -ln.cs[j].y;     // lower elements: x cos - y sin, upper: x cos + y sin
  }
  constexpr int kPer = Lane::kPerWarp;
  const int nq = (d.heads_q + kPer - 1) / kPer, nk = (d.heads_kv + kPer - 1) / kPer;
  // a share of the queries, of the keys and of the values: a key costs about three queries
  const int q0 = nq * part / a.parts, q1 = nq * (part + 1) / a.parts, k0 = nk * part / a.parts,
            k1 = nk * (part + 1) / a.parts;
  const int at = (ln.lane / G) * D + ln.li * 8, step = kPer * D;
  ln.template run<true>(a.q + (int64_t)t * a.ldq + at, a.q_out + (int64_t)t * a.ldqo + at, q0, q1, d.heads_q, step,
                        s_w[0] + ln.li * 8);
  // ---- keys, then values
  const int ng = d.groups, g = ln.li >> 2, k4 = ln.li & 3;
  const bool stored = ln.li < 4 * ng;            // (a last group's lanes past head_dim hold zeros)
  const int code_bytes = 16 * ng;
  auto row_of = [&](int slot) -> uint8_t* {
    if (slot < 0) return nullptr;
    const int page = (int)a.per_page_div.div((uint32_t)slot);
    return reinterpret_cast<uint8_t*>(d.pool) + q4_row(d, page, slot - page * d.per_page);
  };
  // the lane's and its group's error bound, in the largest element of its pairs' groups
  const bool group_err = NORM || (ln.li & ~3) < 2 * half;
  constexpr float kErr = NORM ? kErrNormed : kErrTurned;
  constexpr float kFinest = Elem<E>::kBf16 ? 0x1p-100f : 0x1p-21f, kLargest = Elem<E>::kBf16 ? 31.f * 0x1p123f : 31.f * 0x1p11f;
  const float my_err = NORM || ln.turned ? kErr : 0.f, bump = NORM || ln.turned ? 0.f : 0x1p-15f;
  Exact ex;
  ex.freq = a.freq;
  ex.pos = pos;
  ex.mscale = a.mscale;
  ex.eps = a.eps;
  ex.inv_d = 1.0 / D;
  ex.half = half;
  const float* kw = s_w[1] + ln.li * 8;
  auto heads = [&](const uint16_t* src, uint8_t* row, int j0, int j1, auto is_value) {
    constexpr bool kValue = decltype(is_value)::value;
    for (int jb = j0; jb < j1; jb += kAppendAhead) {
      uint4 raw[kAppendAhead];
#pragma unroll
      for (int j = 0; j < kAppendAhead; ++j)
        raw[j] = ln.live && jb + j < j1 && (jb + j) * kPer + ln.lane / G < d.heads_kv
                     ? *reinterpret_cast<const uint4*>(src + (jb + j) * step)
                     : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < kAppendAhead; ++j) {
        if (jb + j >= j1) break;                 // the same for the whole warp
        const int h = (jb + j) * kPer + ln.lane / G;
        float x[8];
        if (kValue) unpack8<E>(raw[j], x);
        else ln.turn(raw[j], kw, x);
        float hi = max_nan(max3_nan(max3_nan(x[0], x[1], x[2]), x[3], x[4]), max3_nan(x[5], x[6], x[7]));
        float lo = min_nan(min3_nan(min3_nan(x[0], x[1], x[2]), x[3], x[4]), min3_nan(x[5], x[6], x[7]));
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
          lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        }
        const float m = hi >= -lo ? hi : lo, am = fabsf(m);
        float M = copysignf(q4_scale<E>(am), m), top = fminf(am, 3.402823466e38f);
        float inv = M == 0.f ? 0.f : rcp(M) * 8.f;
        if (!kValue) {
          if (!INTER) {                          // (each lane's partner may be in another group)
            float there = __shfl_sync(0xffffffffu, top, ln.partner);
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) there = fmaxf(there, __shfl_xor_sync(0xffffffffu, there, o));
            top = fmaxf(top, there);
          }
          // M may round otherwise where am lies within its error of a number of five bits: in
          // units of its last place, at most 2^24 err / am, and am >= 16 / 17 |M|.  (Below 32
          // units of the finest M its rounding is another: always asked)
          const float err = group_err ? kErr * top : 0.f;
          const uint32_t ulps = (uint32_t)fminf(err * fabsf(inv) * (0x1p21f * 1.07f) + 2.f, 0x1p18f);
          const bool scale = err > 0.f && am <= 3.402823466e38f &&
                             (((__float_as_uint(am) + ulps) & 0x7ffffu) < 2 * ulps || am < 32.f * kFinest ||
                              fabsf(hi + lo) <= 2.f * err);
          if (__any_sync(0xffffffffu, scale)) {
            uint32_t largest = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (scale && fabsf(x[e]) >= am - 2.f * err) largest |= 1u << e;
            const float f = exact_scale<E, NORM, INTER, G>(ex, raw[j], kw, largest);
            if (scale) {
              M = f;
              inv = M == 0.f ? 0.f : rcp(M) * 8.f;
            }
          }
        }
        float k[8], off[8];
        round8(x, inv, kValue ? 0x1p-15f : bump, k, off);
        if (__any_sync(0xffffffffu, am > kLargest)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) k[e] = fminf(k[e], 8.f);
        }
        uint32_t word;
        if (kValue) {
          const uint32_t a0 = nibbles(k[0], k[1], k[2], k[3]), a1 = nibbles(k[4], k[5], k[6], k[7]);
          word = __byte_perm(a0, a1, 0x5410);
        } else {
          const uint32_t a0 = nibbles(k[0], k[2], k[4], k[6]), a1 = nibbles(k[1], k[3], k[5], k[7]);
          word = __byte_perm(a0, a1, 0x5410);
          const float limit = 0.5f - 0x1p-19f - my_err * top * fabsf(inv);    // (t itself: 2^-19.5)
          const float far0 = fmaxf(fmaxf(fabsf(off[0]), fabsf(off[1])), fmaxf(fabsf(off[2]), fabsf(off[3])));
          const float far1 = fmaxf(fmaxf(fabsf(off[4]), fabsf(off[5])), fmaxf(fabsf(off[6]), fabsf(off[7])));
          if (__any_sync(0xffffffffu, my_err > 0.f && fmaxf(far0, far1) > limit)) {
            uint32_t need = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (my_err > 0.f && fabsf(off[e]) > limit) need |= 1u << e;
            word = exact_codes<E, NORM, INTER, G>(ex, raw[j], kw, need, M, word);
          }
        }
        if (stored && row && h < d.heads_kv) {
          uint8_t* codes = row + h * code_bytes;
          if (kValue) {
            reinterpret_cast<uint16_t*>(codes)[2 * k4 * ng + g] = (uint16_t)word;
            reinterpret_cast<uint16_t*>(codes)[(2 * k4 + 1) * ng + g] = (uint16_t)(word >> 16);
          } else {
            reinterpret_cast<uint32_t*>(codes)[k4 * ng + g] = word;
          }
          if (k4 == 0)
            reinterpret_cast<uint16_t*>(row + (int64_t)d.heads_kv * code_bytes)[h * ng + g] = (uint16_t)Elem<E>::from2(M, M);
        }
      }
    }
  };
  heads(a.k + (int64_t)t * a.ldk + at, row_of(ks), k0, k1, std::false_type{});
  heads(a.v + (int64_t)t * a.ldv + at, row_of(vs), k0, k1, std::true_type{});
}

template <class E, bool NORM, bool INTER>
void (*append_kernel(int lanes))(const KvAppendArgs) {
  return lanes == 8 ? kv_q4_append_kernel<E, NORM, INTER, 8> : lanes == 16 ? kv_q4_append_kernel<E, NORM, INTER, 16>
                                                                           : kv_q4_append_kernel<E, NORM, INTER, 32>;
}
template <class E>
void (*append_kernel(bool norm, bool inter, int lanes))(const KvAppendArgs) {
  if (norm) return inter ? append_kernel<E, true, true>(lanes) : append_kernel<E, true, false>(lanes);
  return inter ? append_kernel<E, false, true>(lanes) : append_kernel<E, false, false>(lanes);
}

// ================================================================ read
// Token i: position pos_i of table row row_i, K and V as rows of 16-bit elements.  A warp a
// token; a lane's share of a head of a 4-bit cache is a quarter of each group, 8 elements, one
// load of codes for all groups and one of scales, stored as 16 bytes a group.  Bound: memory,
// the 16-bit rows first, once the three loads in a chain (row and position, page, codes) are
// hidden by other warps.
constexpr int kReadThreads = 256;

// NG: 0, or the groups of a head of a 4-bit cache.
template <class E, int NG>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const __grid_constant__ KvReadArgs a) {
  const KvDev& d = a.kv;
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5);
  if (i >= a.n) return;
  const int row = __ldg(a.row + i), pos = __ldg(a.pos + i);
  if (pos < 0) return;
  const int64_t plane = (int64_t)d.max_rows * d.max_blocks;
  const int b = (int)a.per_page_div.div((uint32_t)pos), in_page = pos - b * d.per_page;
  const bool inside = row >= 0 && row < d.max_rows && b < d.max_blocks;
  int page[2] = {-1, -1};
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (inside && (j ? a.v : a.k)) page[j] = __ldg(d.table + (2 * a.layer + j) * plane + (int64_t)row * d.max_blocks + b);
  const int dim = d.head_dim, width = d.heads_kv * dim;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint16_t* out = j ? a.v : a.k;
    if (!out) continue;
    if ((uint32_t)page[j] >= (uint32_t)d.num_pages) {
      if (lane == 0) report_err(d.error, kErrInvalid);
      continue;
    }
    out += i * (j ? a.ldv : a.ldk);
    if constexpr (NG == 0) {
      const uint16_t* src = d.pool + ((int64_t)page[j] * d.per_page + in_page) * width;
      for (int e = lane * 8; e < width; e += 256) *reinterpret_cast<uint4*>(out + e) = __ldg(reinterpret_cast<const uint4*>(src + e));
    } else {
      const uint8_t* src = reinterpret_cast<const uint8_t*>(d.pool) + q4_row(d, page[j], in_page);
#pragma unroll 2
      for (int u = lane; u < 4 * d.heads_kv; u += 32) {
        const int h = u >> 2, k4 = u & 3;
        uint32_t w[NG], m[(NG + 1) / 2];
        q4_load<NG>(src + (h * 16 + k4 * 4) * NG, src + (d.heads_kv * 16 + h * 2) * NG, w, m);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          uint32_t y[4];
          q4_eight<E, NG>(w, m, g, j == 1, y);
          if (32 * g + 8 * k4 < dim)
            *reinterpret_cast<uint4*>(out + h * dim + 32 * g + 8 * k4) =
                j ? q4_in_order(y) : make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
    }
  }
}

template <class E>
void (*read_kernel(int groups))(const KvReadArgs) {
  switch (groups) {
    case 1: return kv_read_kernel<E, 1>;
    case 2: return kv_read_kernel<E, 2>;
    case 3: return kv_read_kernel<E, 3>;
    case 4: return kv_read_kernel<E, 4>;
    case 5: return kv_read_kernel<E, 5>;
    case 6: return kv_read_kernel<E, 6>;
    case 7: return kv_read_kernel<E, 7>;
    default: return kv_read_kernel<E, 8>;
  }
}

}  // namespace

cudaError_t launch_kv_q4_append(const KvAppendArgs& args, int dtype, int num_sms, cudaStream_t st) {
  KvAppendArgs a = args;
  const int lanes = a.kv.head_dim <= 64 ? 8 : a.kv.head_dim <= 128 ? 16 : 32, per_warp = 32 / lanes;
  // Warps for a token: as many as fill the SMs once, 24 warps each (2084 tokens of 96 heads:
  // 49 us with one, 34 with two; 962: 22 with four).
  const int most = (std::max(a.kv.heads_q, a.kv.heads_kv) + per_warp - 1) / per_warp;
  a.parts = (int)std::max<int64_t>(1, std::min<int64_t>(most, (24 * (int64_t)num_sms + a.T / 2) / a.T));
  const int64_t warps = (int64_t)a.T * a.parts;
  const int grid = (int)((warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
  auto kernel = dtype == 0 ? append_kernel<__half>(a.qw != nullptr, a.interleaved != 0, lanes)
                           : append_kernel<__nv_bfloat16>(a.qw != nullptr, a.interleaved != 0, lanes);
  kernel<<<grid, kAppendThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvReadArgs& a, int dtype, cudaStream_t st) {
  auto kernel = a.kv.groups == 0 ? kv_read_kernel<__half, 0>
                                 : dtype == 0 ? read_kernel<__half>(a.kv.groups) : read_kernel<__nv_bfloat16>(a.kv.groups);
  kernel<<<(unsigned)(((int64_t)a.n + kReadThreads / 32 - 1) / (kReadThreads / 32)), kReadThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace slora
