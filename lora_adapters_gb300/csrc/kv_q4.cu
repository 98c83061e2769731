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
// consecutive elements a lane; a group is four lanes.
//
// Codes are those of the formula in exact arithmetic, not of its fp32 evaluation:
//  - a value that comes straight from 16 bits has at most 11 significant bits, a
//    border (2n + 1) M / 16 at most 9, so the two are equal or at least 2^-11 of the
//    border apart.  t = 8 x / M evaluated with an error below 2^-18 and raised by
//    2^-15 then rounds to the right integer, ties upwards;
//  - a normed or rotated key has an error of at most kErr times the head's largest
//    element (cosine and sine 2^-22, two products and a sum; the pair's length is at
//    most sqrt(2) times that element; the norm's factor 2^-21).  Where that could
//    change a code, M's rounding or the choice between the two signs, the warp
//    works the elements in question out again in fp64 (requantise: about one head in
//    200).
constexpr int kAppendThreads = 256;
constexpr float kErr = 0x1p-19f;

// What requantise needs of a lane.
struct Exact {
  const uint64_t* freq;
  int64_t pos;
  float mscale, eps;
  int head_dim, half;            // half: lanes between the halves of the half layout
};

// The group's codes (packed as K's) and M in fp64 where they are in question: `need`
// has a bit for each of the lane's elements, all of them set where M is.  By a whole
// warp; r: the lane's raw elements, w: its weights.
template <class E, bool NORM, bool INTER, int G>
__device__ __noinline__ uint2 requantise(const Exact ex, uint4 r, const float* w, uint32_t need, bool scale_too, float M,
                                         uint32_t word) {
  const int lane = threadIdx.x & 31, li = lane & (G - 1);
  const int pl = li < ex.half ? li + ex.half : li - ex.half;
  const bool turned = li < 2 * ex.half;
  const int partner = (lane & ~(G - 1)) | (turned ? pl : li);
  float own[8], other[8];
  unpack8<E>(r, own);
  if (!INTER) {
    uint4 o;
    o.x = __shfl_sync(0xffffffffu, r.x, partner);
    o.y = __shfl_sync(0xffffffffu, r.y, partner);
    o.z = __shfl_sync(0xffffffffu, r.z, partner);
    o.w = __shfl_sync(0xffffffffu, r.w, partner);
    unpack8<E>(o, other);
  }
  double rs = 1.0;
  if (NORM) {
    double ss = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += (double)own[e] * own[e];
#pragma unroll
    for (int o = G >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    rs = 1.0 / sqrt(ss / ex.head_dim + (double)ex.eps);
  }
  double x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = own[e];
    if (!__any_sync(0xffffffffu, (need >> e) & 1)) continue;
    const int partner_e = INTER ? e ^ 1 : e;
    double a = own[e], b = INTER ? own[partner_e] : other[e];
    if (NORM) {                                    // (x w exactly: equal magnitudes stay equal)
      a = a * w[e] * rs;
      b = b * (INTER ? w[partner_e] : w[((turned ? pl : li) - li) * 8 + e]) * rs;
    }
    x[e] = a;
    if (turned) {
      const int pi = INTER ? li * 4 + e / 2 : (li < ex.half ? li : pl) * 8 + e;
      double c, s;
      sincospi((double)(int64_t)((uint64_t)ex.pos * ex.freq[pi]) * 0x1p-63, &s, &c);
      const bool first = INTER ? (e & 1) == 0 : li < ex.half;
      x[e] = (a * c + (first ? -b : b) * s) * (double)ex.mscale;
    }
  }
  if (__any_sync(0xffffffffu, scale_too)) {
    double hi = x[0], lo = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
      hi = fmax(hi, x[e]);
      lo = fmin(lo, x[e]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      hi = fmax(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      lo = fmin(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    if (scale_too && M == M) {                     // (a group that is not finite stays so)
      const double m = hi >= -lo ? hi : lo;
      M = copysignf(q4_scale<E>(__double2float_ru(fabs(m))), (float)m);   // (upwards, as M itself)
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if ((need >> e) & 1) {
      const double k = M == 0.f ? 0.0 : fmin(fmax(floor(8.0 * x[e] / (double)M + 0.5), -7.0), 8.0);
      const int at = 16 * (e & 1) + 4 * (e >> 1);
      word = (word & ~(15u << at)) | (uint32_t)((int)k + 7) << at;
    }
  }
  return make_uint2(word, __float_as_uint(M));
}

__device__ __forceinline__ uint32_t nibbles(float a, float b, float c, float e) {   // of codes k, the first lowest
  return __float_as_uint(fmaf(fmaf(fmaf(e, 16.f, c), 16.f, b), 16.f, a) + (8388608.f + 0x7777));
}
// The codes k of x (inv = 8 / M, bump: by how much 8 x / M is raised), and in d how far
// they are from it before they are held within -7 .. 8.
__device__ __forceinline__ void round8(const float (&x)[8], float inv, float bump, float (&k)[8], float (&d)[8]) {
  constexpr float kInt = 12582912.f;               // 1.5 * 2^23: adding it rounds to an integer
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = fmaf(x[e], inv, bump), r = (t + kInt) - kInt;
    d[e] = r - t;
    k[e] = fminf(fmaxf(r, -7.f), 8.f);
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
    for (int i = tid; i < 2 * D; i += kAppendThreads)
      s_w[i >= D][i >= D ? i - D : i] = Elem<E>::to(i >= D ? a.kw[i - D] : a.qw[i]);
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
  const int iters = nq + 2 * nk, i0 = iters * part / a.parts, i1 = iters * (part + 1) / a.parts;
  const int at = (ln.lane / G) * D + ln.li * 8, step = kPer * D;
  ln.template run<true>(a.q + (int64_t)t * a.ldq + at, a.q_out + (int64_t)t * a.ldqo + at, i0, min(i1, nq), d.heads_q, step,
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
  // the lane's and its group's error bound, in the head's largest element
  const bool group_err = NORM || (ln.li & ~3) < 2 * half;
  const float my_err = NORM || ln.turned ? kErr : 0.f, bump = NORM || ln.turned ? 0.f : 0x1p-15f;
  Exact ex;
  ex.freq = a.freq;
  ex.pos = pos;
  ex.mscale = a.mscale;
  ex.eps = a.eps;
  ex.head_dim = D;
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
        float M = copysignf(q4_scale<E>(am), m);
        const float inv = M == 0.f ? 0.f : 8.f / M;
        float k[8], off[8];
        round8(x, inv, kValue ? 0x1p-15f : bump, k, off);
        uint32_t word;
        if (kValue) {
          const uint32_t a0 = nibbles(k[0], k[1], k[2], k[3]), a1 = nibbles(k[4], k[5], k[6], k[7]);
          word = __byte_perm(a0, a1, 0x5410);
        } else {
          const uint32_t a0 = nibbles(k[0], k[2], k[4], k[6]), a1 = nibbles(k[1], k[3], k[5], k[7]);
          word = __byte_perm(a0, a1, 0x5410);
          float top = am;                        // the head's largest element
#pragma unroll
          for (int o = 4; o < G; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const float err = my_err * top, m_err = group_err ? kErr * top : 0.f;
          const float limit = 0.5f - 0x1p-18f - err * fabsf(inv);
          const float far0 = fmaxf(fmaxf(fabsf(off[0]), fabsf(off[1])), fmaxf(fabsf(off[2]), fabsf(off[3])));
          const float far1 = fmaxf(fmaxf(fabsf(off[4]), fabsf(off[5])), fmaxf(fabsf(off[6]), fabsf(off[7])));
          const bool code = my_err > 0.f && fmaxf(far0, far1) > limit;
          const bool scale = m_err > 0.f && am <= 3.402823466e38f &&
                             (q4_scale<E>(am + m_err) != q4_scale<E>(fmaxf(am - m_err, 0.f)) || fabsf(hi + lo) <= 2.f * m_err);
          if (__any_sync(0xffffffffu, code || scale)) {
            uint32_t need = scale ? 0xffu : 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (my_err > 0.f && fabsf(off[e]) > limit) need |= 1u << e;
            const uint2 f = requantise<E, NORM, INTER, G>(ex, raw[j], kw, need, scale, M, word);
            word = f.x;
            M = __uint_as_float(f.y);
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
  heads(a.k + (int64_t)t * a.ldk + at, row_of(ks), max(i0 - nq, 0), min(i1 - nq, nk), std::false_type{});
  heads(a.v + (int64_t)t * a.ldv + at, row_of(vs), max(i0 - nq - nk, 0), i1 - nq - nk, std::true_type{});
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
// Token i: position pos_i of table row row_i, K and V as rows of 16-bit elements.
constexpr int kReadThreads = 256;

template <class E, bool Q4>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const __grid_constant__ KvReadArgs a) {
  const KvDev& d = a.kv;
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kReadThreads / 32), plane = (int64_t)d.max_rows * d.max_blocks;
  const int width = d.heads_kv * d.head_dim;
  for (int64_t u = (int64_t)blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5); u < 2 * (int64_t)a.n; u += warps) {
    const int i = (int)(u >> 1), j = (int)(u & 1);
    uint16_t* out = j ? a.v : a.k;
    const int row = __ldg(a.row + i), pos = __ldg(a.pos + i);
    if (!out || pos < 0) continue;
    int page = -1, in_page = 0;
    if (row >= 0 && row < d.max_rows) {
      const int b = (int)a.per_page_div.div((uint32_t)pos);
      in_page = pos - b * d.per_page;
      if (b < d.max_blocks) page = __ldg(d.table + (2 * a.layer + j) * plane + (int64_t)row * d.max_blocks + b);
    }
    if ((uint32_t)page >= (uint32_t)d.num_pages) {
      if (lane == 0) report_err(d.error, kErrInvalid);
      continue;
    }
    out += i * (j ? a.ldv : a.ldk);
    if (!Q4) {
      const uint16_t* src = d.pool + ((int64_t)page * d.per_page + in_page) * width;
      for (int e = lane * 8; e < width; e += 256) *reinterpret_cast<uint4*>(out + e) = *reinterpret_cast<const uint4*>(src + e);
    } else {
      const uint8_t* src = reinterpret_cast<const uint8_t*>(d.pool) + q4_row(d, page, in_page);
      const int ng = d.groups, words = 4 * ng;     // 8 elements each
      for (int w = lane; w < words * d.heads_kv; w += 32) {
        const int h = w / words, li = w - h * words, g = li >> 2, k4 = li & 3;
        if (li * 8 >= d.head_dim) continue;
        const uint8_t* codes = src + h * 16 * ng;
        const float M = Elem<E>::to(reinterpret_cast<const uint16_t*>(src + (int64_t)d.heads_kv * 16 * ng)[h * ng + g]);
        float x[8];
        if (j) {
          const uint32_t c = reinterpret_cast<const uint16_t*>(codes)[2 * k4 * ng + g] |
                             (uint32_t)reinterpret_cast<const uint16_t*>(codes)[(2 * k4 + 1) * ng + g] << 16;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = q4_value(c >> (4 * e) & 15, M);
        } else {
          const uint32_t c = reinterpret_cast<const uint32_t*>(codes)[k4 * ng + g];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = q4_value(c >> (16 * (e & 1) + 4 * (e >> 1)) & 15, M);
        }
        *reinterpret_cast<uint4*>(out + h * d.head_dim + li * 8) = pack8<E>(x);
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_q4_append(const KvAppendArgs& args, int dtype, int num_sms, cudaStream_t st) {
  KvAppendArgs a = args;
  const int lanes = a.kv.head_dim <= 64 ? 8 : a.kv.head_dim <= 128 ? 16 : 32, per_warp = 32 / lanes;
  const int iters = (a.kv.heads_q + per_warp - 1) / per_warp + 2 * ((a.kv.heads_kv + per_warp - 1) / per_warp);
  a.parts = std::max(1, std::min(iters, 16 * num_sms / a.T));
  const int64_t warps = (int64_t)a.T * a.parts;
  const int grid = (int)((warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
  auto kernel = dtype == 0 ? append_kernel<__half>(a.qw != nullptr, a.interleaved != 0, lanes)
                           : append_kernel<__nv_bfloat16>(a.qw != nullptr, a.interleaved != 0, lanes);
  kernel<<<grid, kAppendThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvReadArgs& a, int dtype, int num_sms, cudaStream_t st) {
  const int64_t ctas = (2 * (int64_t)a.n + kReadThreads / 32 - 1) / (kReadThreads / 32);
  const int grid = (int)std::min<int64_t>(ctas, 16 * num_sms);
  auto kernel = a.kv.groups == 0 ? kv_read_kernel<__half, false>
                                 : dtype == 0 ? kv_read_kernel<__half, true> : kv_read_kernel<__nv_bfloat16, true>;
  kernel<<<grid, kReadThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace slora
