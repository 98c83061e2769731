// slora_kv_attend for few query rows (decode) over a cache held in 4 bits: the split
// over the cache's length and the products of attend.cu, from codes.
//
// With codes c = k + 7 and a scale M for every token and group of 32 elements
// (kv_q4.cuh), scores and results are
//     s_j = q . k_j = sum_g M^K_jg / 8 (sum_e q_e c_e - 7 sum_e q_e),   e in group g,
//     o_e = sum_j p_j v_je = 1/8 (sum_j (p_j M^V_jg) c_je - 7 sum_j p_j M^V_jg),
// so that the matrix operands are the codes themselves:
//  - a code in the low bits of a 16-bit word is the fp16 number c 2^-24 (subnormal), four
//    bits further up 16 c 2^-24: one AND of a loaded word is an operand register, for
//    both storage types.  The two positions go to products of their own, and the factor
//    16 into Q or the result;
//  - K's scale multiplies a group's accumulator, a pair of steps of the sum over the
//    head; the offset 7 sum(q) is the accumulator's first value.  Queries are scaled by
//    a power of two to below 2^14 (heads above 128: 2^13) first, which fp16's exponents hold
//    for bf16 too (bits below 2^-24, or 2^-23, of a row's largest element are lost);
//  - V's scale goes into the weights.  bf16 caches have every weight p in one fp16 part:
//    2^-11 of it, and as much for its product with M 2^(7 - E) (|M| < 2^E so far), are an
//    eighth of the rounding of a result each, of the element itself (the offset's sum is of
//    the rounded products too).  fp16 caches have two, p = hi + lo, and hi M is again two
//    parts, a product and its exact remainder.  Columns of the product that have no row
//    (fewer than 8 query rows) take other groups' weights: RT rows times 8 / RT groups fill
//    them, and a token's weights are worked out that many times less often;
//  - each unit's result starts from zero and is added to the running one in fp32: with
//    codes that are never negative, a running sum in the tensor core would lose bits
//    to its truncation.
//
// Bound: the latency of a unit's steps, which follow each other in every warp (barrier, scores,
// maximum, weights, results), with three warps a scheduler to hide it.  Per 32 tokens of
// a head of 128 there are 4,608 bytes, 196 cycles of an SM's share of the memory, against 715
// (two rows, weights in two parts) or 820 (eight rows, in one) instructions of a warp, 180 or 205
// cycles of its issue slots, of which 53 and 62 % are taken; the integer and logic pipe is
// busy 46 and 50 % of the time, and results of a fixed latency are what warps wait for most.
// Measured: 256 requests of 8 to 640 tokens, 32 heads of 128, 114 us (3.4 TB/s of codes and
// scales; the copies alone 70); 128 requests of 17 to 8192 tokens, 40 heads on 8, 162 us (3.8
// TB/s; 105).  The times beside the rules below are single calls' over a cold cache, 115 and 165
// for these two.
#include <type_traits>

#include "attend.cuh"
#include "kv_q4.cuh"

namespace slora {
namespace {

// Warps of a CTA: one for each of the neighbouring key heads that it works on, at most
// kMaxAbreast; and as many CTAs an SM as make q4_warps.
constexpr int kMaxAbreast = 6;
__host__ __device__ constexpr int q4_rounded(int ng) { return ng <= 2 ? 2 : ng <= 4 ? 4 : 8; }
// An SM: 168 or 255 registers a thread.  (16 of up to 4 groups, 128 registers: they spill,
// 184 us instead of 165 for 128 requests of 17 to 8192 tokens, 40 heads on 8.)
constexpr int q4_warps(int ng) { return ng <= 4 ? 12 : 6; }

__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t y;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
  return y;
}
__device__ __forceinline__ uint32_t h2_neg(uint32_t a) {
  uint32_t y;
  asm("neg.f16x2 %0, %1;" : "=r"(y) : "r"(a));
  return y;
}
__device__ __forceinline__ const uint8_t* shfl_ptr(const uint8_t* p, int src) {
  return reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), src));
}
// 16 bytes global -> shared, asynchronously, past the first-level cache; bytes = 0: zeros,
// nothing is read.
__device__ __forceinline__ void cp_async(uint32_t dst, const uint8_t* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// N consecutive words of shared memory (N = 1, 2, 4, 8), at a multiple of min(4 N, 16) bytes.
template <int N>
__device__ __forceinline__ void lds(uint32_t at, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "r"(at + 4 * i));
  }
}
__device__ __forceinline__ uint32_t lds_half(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}
template <int N>
__device__ __forceinline__ void sts(uint32_t at, const uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 4 * i), "r"(w[i]) : "memory");
}

// A CTA's ring of units in shared memory.  Of a unit: K's codes [head][token][16 NG bytes];
// V's, the same, with 16-byte pieces exchanged so that the four tokens that a warp reads at
// a time lie in different banks; K's scales and V's, [token][all heads', from the last
// multiple of 16 bytes before them].
template <int NG>
struct Ring {
  static constexpr int kUnit = NG <= 4 ? 32 : 16;      // kv_q4_unit
  // 128 requests of 17 to 2048 tokens, 16 heads of 160: 235 us with 2 and with 3; of 192 230
  // and 229; of 256 233 and 222 (8 key heads of two rows 125 and 119, of 224 145 and
  // 154).  256 requests of 8 to 640, 32 heads of 128: 115 and 117.
  static constexpr int kStages = NG == 8 ? 3 : 2;
  static constexpr int kCodes = kUnit * 16 * NG;       // of a head
  static constexpr int kRows = kUnit * 16 + 16;        // where a unit's rows begin, which are there, the block of heads
  // where 16-byte piece p of token t of V lies
  static __device__ __forceinline__ int v_piece(int t, int p) {
    constexpr int kPer = NG == 8 ? 1 : 8 / NG;         // tokens of 128 bytes
    return (t / kPer) * 128 + ((((t % kPer) * NG + p) ^ (NG == 2 ? 2 * ((t >> 2) & 1) : 2 * ((t >> 1) & 3))) << 4);
  }
};
// Bytes that hold the scales of `heads` neighbouring heads of a token, wherever they begin.
__host__ __device__ __forceinline__ int scale_bytes(int heads, int ng) {
  const int n = heads * 2 * ng, step = n & -n;         // they begin at multiples of it
  return n % 16 ? (n + 31 - step) / 16 * 16 : n;
}
template <int NG>
__host__ __device__ __forceinline__ int stage_bytes(int heads, int ng) {
  return 2 * (heads * Ring<NG>::kCodes + Ring<NG>::kUnit * scale_bytes(heads, ng));
}
template <int NG>
__host__ __device__ __forceinline__ int ring_bytes(int heads, int ng) {
  return Ring<NG>::kStages * stage_bytes<NG>(heads, ng) + 4 * Ring<NG>::kRows + heads * Ring<NG>::kUnit * 2 * NG;
}

// D = A B + C.  Not volatile: the compiler may place products that do not depend on each
// other between those that do.
__device__ __forceinline__ void mma_h(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1, float c0, float c1, float c2, float c3) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// NC: groups of a head, NG: rounded up to 2, 4 or 8; RT: rows that have columns of their own.
template <class E, int NC, int RT, bool CAP>
__global__ void __launch_bounds__(kMaxAbreast * 32, q4_warps(NC) / kMaxAbreast)
kv_q4_decode_kernel(const __grid_constant__ KvAttendArgs a) {
  constexpr int NG = q4_rounded(NC), ng = NC, W = NG / 2;      // W: words of a token's scales
  constexpr bool FULL = NC == NG;
  constexpr int GC = 8 / RT;        // groups whose weights lie side by side
  constexpr int PASS = (NC + GC - 1) / GC;             // sets of weights a token has
  constexpr int NR = RT == 8 ? 2 : 1;                  // rows of a lane
  using R = Ring<NG>;
  constexpr int UNIT = R::kUnit, NS = UNIT / 16;
  // Queries are scaled to below 2^(kQTop + 1): a group's product with codes is then at most 2^-2 (2^-3),
  // and the sum over 4 (8) groups times M, which reaches 31 2^123, below 2^128
  constexpr int kQTop = NG == 8 ? 12 : 13;
  constexpr int NO = RT == 2 ? NG / 2 : NC;            // groups of a lane's results
  // Parts of a weight.  256 requests of 8 to 640 tokens, 32 heads of fp16: 115 us with two,
  // 107 with one, which costs the result's last bit; 128 requests of 17 to 8192, 40 heads
  // on 8 of bf16: 182 and 165 us.
  constexpr int kParts = Elem<E>::kBf16 ? 1 : 2;
  constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
  constexpr uint32_t kNotFinite = Elem<E>::kBf16 ? 0x7f80u : 0x7c00u;    // infinity's bits
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const KvDev& d = a.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // a group of CTAs takes the same units of hbw neighbouring heads, one head a warp
  const int heads = blockDim.x >> 5, hbw = a.hbw, blocks = d.heads_kv / hbw, ctas = hbw / heads;
  const int grp = blockIdx.x / ctas, hsub0 = (blockIdx.x - grp * ctas) * heads, hsub = hsub0 + warp;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem_raw);
  const int stage_size = stage_bytes<NG>(heads, ng), scale_size = scale_bytes(heads, ng);
  const int at_v = heads * R::kCodes, at_ks = 2 * at_v, at_vs = at_ks + UNIT * scale_size;   // in a stage
  const DecSplit sp = dec_split(__ldg(d.dec_off + a.R), blocks, gridDim.x / ctas);
  const int64_t u = grp * sp.run, u1 = min(sp.total, u + sp.run);
  const int dim = d.head_dim, P = d.per_page, group = d.heads_q / d.heads_kv;
  const int kk = lane & 3, nn = lane >> 2;
  const int64_t plane = (int64_t)d.max_rows * d.max_blocks;
  const float sc = kLog2e * a.scale, cap_t = a.cap_t, cap2 = a.cap2;
  if (u >= u1) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  int left = (int)min(u1 - u, (int64_t)0x7fffffff);

  // Units are on their way to shared memory while the ones before them are multiplied, from
  // one segment into the next; their pages are looked up one ahead of that.
  struct {
    int left, r, hb, rt, c;        // units left; request, head block, row tile, unit of the segment
    int n, tiles, len;             // units of a segment, row tiles, tokens of the request
    const int32_t* tab;            // the request's K pages
  } f;
  auto f_open = [&](const int4& rq) {
    f.len = rq.z;
    f.n = (rq.z + UNIT - 1) / UNIT;
    f.tiles = (rq.y * group + RT - 1) / RT;
    f.tab = d.table + 2 * a.layer * plane + (int64_t)dbg_index(rq.w, d.max_rows, d.error) * d.max_blocks;
  };
  auto no_units = [&](const int4& rq) {
    return rq.y == 0 || (a.tpt > 0 && (int64_t)rq.y * group > kKvChunkRows);
  };
  {
    f.left = left;
    f.r = find_request(d.dec_off, a.R, u, blocks);
    const int4 rq = __ldg(d.req + f.r);
    f_open(rq);
    const int64_t in_req = u - (int64_t)__ldg(d.dec_off + f.r) * blocks;
    const int seg = (int)(in_req / f.n);
    f.c = (int)(in_req - (int64_t)seg * f.n);
    f.hb = seg / f.tiles;
    f.rt = seg - f.hb * f.tiles;
  }
  int r = f.r, hb = f.hb, rt = f.rt, c0 = f.c;          // the segment that is multiplied
  // A unit's rows are looked up by one warp, in turn, and left in shared memory for the others:
  // asked for one unit before they are needed, written a barrier before.  Of a token past
  // the request's length, or without a page, nothing is read: its codes and scales are
  // zeros, and its scores are masked.
  struct Pages {
    int k, v, in_page;             // of token lane % UNIT, in_page -1: none
  };
  auto fetch = [&](Pages& p, bool mine) -> int {         // the unit's block of heads
    p.in_page = -1;
    if (f.left == 0) return 0;
    --f.left;
    if (f.c == f.n) {
      f.c = 0;
      if (++f.rt == f.tiles) {
        f.rt = 0;
        if (++f.hb == blocks) {
          f.hb = 0;
          int4 rq;
          do rq = __ldg(d.req + ++f.r);
          while (no_units(rq));
          f_open(rq);
        }
      }
    }
    const int j = f.c++ * UNIT + (lane & (UNIT - 1));
    if (mine && j < f.len) {
      const int b = (int)a.per_page_div.div((uint32_t)j);
      p.in_page = j - b * P;
      p.k = __ldg(f.tab + b);
      p.v = __ldg(f.tab + plane + b);
    }
    return f.hb;
  };
  bool missing = false;
  const uint32_t rows_at = ring + R::kStages * stage_size;
  auto publish = [&](const Pages& p, int block, uint32_t slot) {
    const bool token = p.in_page >= 0;
    const bool ok = token && (uint32_t)p.k < (uint32_t)d.num_pages && (uint32_t)p.v < (uint32_t)d.num_pages;
    missing |= token && !ok;
    const int kp = ok ? p.k : 0, vp = ok ? p.v : 0, at = ok ? p.in_page : 0;
    const uint8_t* pool = reinterpret_cast<const uint8_t*>(d.pool);
    const uint32_t to = rows_at + slot * R::kRows, valid = __ballot_sync(0xffffffffu, ok);
    asm volatile("st.shared.v2.u64 [%0], {%1, %2};" ::"r"(to + (lane & (UNIT - 1)) * 16), "l"(pool + q4_row(d, kp, at)),
                 "l"(pool + q4_row(d, vp, at))
                 : "memory");
    if (lane == 0)
      asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(to + UNIT * 16), "r"(valid), "r"(block) : "memory");
  };
  const int scale_at = d.heads_kv * 16 * ng;
  // This thread's part of a unit's copies: piece `piece` of head `p_head`'s codes, of the tokens
  // p_token, p_token + 32 / NG, ...  A token's pieces of all heads are consecutive threads'
  const int p_token = tid / (heads * NG), p_head = tid % (heads * NG) / NG, piece = tid % NG;
  const uint32_t to_k = ring + p_head * R::kCodes + p_token * 16 * NG + piece * 16,
                 to_v = ring + at_v + p_head * R::kCodes + R::v_piece(p_token, piece);
  // Copies the unit whose rows are in `slot` to a stage of the ring; the tokens with both
  // rows, a bit each.
  auto issue = [&](uint32_t slot, uint32_t stage) -> uint32_t {
    const uint32_t rows = rows_at + slot * R::kRows, to = stage * stage_size;
    uint32_t vh[2];
    lds<2>(rows + UNIT * 16, vh);
    const uint32_t valid = vh[0];
    const int head0 = vh[1] * hbw + hsub0, in_row = ((head0 + p_head) * ng + piece) * 16;
    auto codes = [&](auto all) {
      constexpr bool kAll = decltype(all)::value;
#pragma unroll
      for (int x = 0; x < UNIT * NG / 32; ++x) {
        const int t = p_token + x * (32 / NG);
        const uint8_t *k, *v;
        asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(k), "=l"(v) : "r"(rows + t * 16));
        const uint32_t bytes = kAll || (valid >> t & 1) ? 16 : 0;
        if (FULL || piece < ng) {
          cp_async(to + to_k + x * 512, k + in_row, bytes);
          // (tokens 32 / NG apart lie 512 bytes apart; NG = 8: with another exchange of the pieces)
          cp_async(to + (NG == 8 ? to_v ^ (x & 1) << 6 : to_v) + x * 512, v + in_row, bytes);
        }
      }
    };
    if (valid == ~0u) codes(std::true_type{});
    else codes(std::false_type{});
    // scales: K's pieces, then V's, one a warp (UNIT = 16: two) for all tokens
    const int s_row = scale_at + head0 * 2 * ng, pieces = ((s_row & 15) + heads * 2 * ng + 15) >> 4;
    const int own = lane & (UNIT - 1);
    for (int i = tid / UNIT; i < 2 * pieces; i += heads * 32 / UNIT) {
      const bool v = i >= pieces;
      const int from = (v ? i - pieces : i) * 16;
      const uint8_t* row;
      asm volatile("ld.shared.u64 %0, [%1];" : "=l"(row) : "r"(rows + own * 16 + (v ? 8 : 0)));
      cp_async(ring + to + (v ? at_vs : at_ks) + own * scale_size + from, row + (s_row & ~15) + from,
               valid >> own & 1 ? 16 : 0);
    }
    cp_commit();
    return valid;
  };
  // Scales of a token from the ring.
  auto token_scales = [&](uint32_t at, uint32_t (&w)[W]) {
    if constexpr (FULL) {
      lds<W>(at, w);
    } else {                         // perhaps from the middle of a word on
      uint32_t v[W] = {};
#pragma unroll
      for (int i = 0; i < (NC + 1) / 2; ++i) {
        uint32_t x[1];
        lds<1>((at & ~3u) + 4 * i, x);
        v[i] = x[0];
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        w[i] = at & 2 ? v[i] >> 16 | (i + 1 < W ? v[i + 1] << 16 : 0u) : v[i];
        if (2 * i >= NC) w[i] = 0;
        if (2 * i + 1 == NC) w[i] &= 0xffffu;
      }
    }
  };
  // the values' scales as fp16 times 2^(7 - E), a warp's own
  const uint32_t my_scales = rows_at + 4 * R::kRows + warp * (UNIT * 2 * NG);
  // units 0 .. kAhead published, all but the last of them on their way, the next looked up
  constexpr int kAhead = R::kStages - 1;
  Pages next;
  int block;
  {
    Pages first[kAhead + 1];
    int first_block[kAhead + 1];
#pragma unroll
    for (int x = 0; x <= kAhead; ++x) first_block[x] = fetch(first[x], warp == x % heads);
    block = fetch(next, warp == (kAhead + 1) % heads);
#pragma unroll
    for (int x = 0; x <= kAhead; ++x)
      if (warp == x % heads) publish(first[x], first_block[x], x);
  }
  __syncthreads();
  uint32_t valid[kAhead + 1], stage = 0, unit = 0;
#pragma unroll
  for (int x = 0; x < kAhead; ++x) valid[x] = issue(x, x);
  int turn = (kAhead + 1) % heads;           // the warp that looked unit + kAhead + 1 up

  while (left > 0) {
    int4 rq = __ldg(d.req + r);
    while (no_units(rq)) rq = __ldg(d.req + ++r);
    const int len = rq.z, q0 = rq.x, rows = rq.y * group;
    const int nchunk = (len + UNIT - 1) / UNIT, tiles = (rows + RT - 1) / RT;
    const int c1 = min(nchunk, c0 + left);
    const int hk = hb * hbw + hsub;
    const int ctx = len - rq.y;
    // ---- this tile's queries: column n has row n / GC, (token, head of the group).  Eight
    // elements of every group a lane, in the order of K's codes
    uint32_t qf[NC][4];
    float c_first[NC][NR], fac[NR];
    {
      const int row = rt * RT + nn / GC;
      const bool in = row < rows;
      const uint16_t* src = a.q + (int64_t)dbg_index(q0 + (in ? row / group : 0), a.T, d.error) * a.ldq +
                            (int64_t)(hk * group + (in ? row % group : 0)) * dim;
      float top = 0.f;
      uint4 raw[NC];
#pragma unroll
      for (int g = 0; g < NC; ++g) {
        const int e = 32 * g + 8 * kk;
        raw[g] = make_uint4(0, 0, 0, 0);
        if (in && e < dim) raw[g] = *reinterpret_cast<const uint4*>(src + e);
        float x[8];
        unpack8<E>(raw[g], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^e <= top < 2^(e + 1); e = -100 where it is less
      const int e = max((int)(__float_as_uint(top) >> 23) - 127, -100);
      const float up = __uint_as_float((uint32_t)(127 + kQTop - e) << 23);   // (infinity, NaN: e = 128)
      const float size = __uint_as_float((uint32_t)(127 + min(e, 127)) << 23);
      // 2^(21 - kQTop + e), kept finite: a product of 0 has the score 0 for queries of every size
      constexpr float kDown = 1 << (21 - kQTop);
      const float down = fminf(CAP ? size * kDown : size * sc * kDown, 0x1.fffffep127f);
#pragma unroll
      for (int g = 0; g < NC; ++g) {
        float x[8], sum = 0.f;
        unpack8<E>(raw[g], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] *= up;
          sum += x[i];
        }
        qf[g][0] = Elem<__half>::from2(x[0], x[1]);
        qf[g][1] = Elem<__half>::from2(x[4], x[5]);
        qf[g][2] = Elem<__half>::from2(x[2] * 0.0625f, x[3] * 0.0625f);
        qf[g][3] = Elem<__half>::from2(x[6] * 0.0625f, x[7] * 0.0625f);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= -7.f * 0x1p-24f;
#pragma unroll
        for (int x2 = 0; x2 < NR; ++x2) c_first[g][x2] = __shfl_sync(0xffffffffu, sum, (2 * kk + x2) * 4);
      }
#pragma unroll
      for (int x2 = 0; x2 < NR; ++x2) fac[x2] = __shfl_sync(0xffffffffu, down, (2 * kk + x2) * 4);
    }
    // keys that this lane's rows may see: positions below lim
    const int my_row = rt * RT + 2 * kk / GC;
    int lim[NR];
#pragma unroll
    for (int x = 0; x < NR; ++x) lim[x] = ctx + min(my_row + x, rows - 1) / group + 1;
    const int lim_first = ctx + rt * RT / group + 1;       // of the tile's first row

    // results: elements 32 g + 4 nn + i of the lane's groups and rows; sums of p M a group
    float o[NO][NR][4], lg[NO][NR], m[NR], l[NR];
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      m[x] = -INFINITY;
      l[x] = 0.f;
#pragma unroll
      for (int g = 0; g < NO; ++g) {
        lg[g][x] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[g][x][i] = 0.f;
      }
    }
    const int at_scales = ((scale_at + (hb * hbw + hsub0) * 2 * ng) & 15) + warp * 2 * ng;     // of the head, in a token's
    // E: every |M| so far is below 2^E.  Begins where the smallest M (bf16 2^-100, fp16 2^-21) is held exactly
    int top_m = Elem<E>::kBf16 ? -100 : -8;

    for (int c = c0; c < c1; ++c) {
      cp_wait<kAhead - 1>();
      __syncthreads();             // every thread's copies of this unit have landed, the last unit's are read
      const uint32_t here = ring + stage * stage_size, my_k = here + warp * R::kCodes, my_v = my_k + at_v;
      valid[kAhead] = issue((unit + kAhead) & 3, stage == 0 ? kAhead : stage - 1);
      if (warp == turn) publish(next, block, (unit + kAhead + 1) & 3);
      turn = turn == heads - 1 ? 0 : turn + 1;
      block = fetch(next, warp == turn);
      ++unit;
      // ---- scores of tokens nn + 8 x
      float s[2 * NS][NR];
#pragma unroll
      for (int x = 0; x < 2 * NS; x += 2) {
        uint32_t kf[2][NG], km[2][W];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int t = nn + 8 * (x + z);
          if constexpr (FULL) {
            lds<NG>(my_k + t * 16 * NG + kk * 4 * NG, kf[z]);
          } else {
#pragma unroll
            for (int g = 0; g < NC; ++g) {
              uint32_t w[1];
              lds<1>(my_k + t * 16 * NG + (kk * NC + g) * 4, w);
              kf[z][g] = w[0];
            }
          }
          token_scales(here + at_ks + t * scale_size + at_scales, km[z]);
        }
#pragma unroll
        for (int y = 0; y < NR; ++y) s[x][y] = s[x + 1][y] = 0.f;
        float acc[NC][4];
#pragma unroll
        for (int g = 0; g < NC; ++g) {
          const uint32_t w0 = kf[0][g], w1 = kf[1][g], h0 = w0 >> 8, h1 = w1 >> 8;
          mma_h(acc[g], w0 & kLow, w1 & kLow, h0 & kLow, h1 & kLow, qf[g][0], qf[g][1], c_first[g][0], c_first[g][NR - 1],
                c_first[g][0], c_first[g][NR - 1]);
        }
#pragma unroll
        for (int g = 0; g < NC; ++g) {
          const uint32_t w0 = kf[0][g], w1 = kf[1][g], h0 = w0 >> 8, h1 = w1 >> 8;
          mma_h(acc[g], w0 & kHigh, w1 & kHigh, h0 & kHigh, h1 & kHigh, qf[g][2], qf[g][3], acc[g][0], acc[g][1], acc[g][2],
                acc[g][3]);
        }
#pragma unroll
        for (int g = 0; g < NC; ++g) {
          const float2 M0 = Elem<E>::to2(km[0][g / 2]), M1 = Elem<E>::to2(km[1][g / 2]);
#pragma unroll
          for (int y = 0; y < NR; ++y) {
            s[x][y] = fmaf(acc[g][y], g & 1 ? M0.y : M0.x, s[x][y]);
            s[x + 1][y] = fmaf(acc[g][2 + y], g & 1 ? M1.y : M1.x, s[x + 1][y]);
          }
        }
      }
      // (before masks and maximum: -infinity times a factor that is 0 for a tiny scale would be no
      // number, and of a large score the maximum's rounding would be left beside it)
#pragma unroll
      for (int y = 0; y < NR; ++y)
#pragma unroll
        for (int x = 0; x < 2 * NS; ++x) {
          s[x][y] *= fac[y];
          if (CAP) s[x][y] = capped<true>(s[x][y], sc, cap_t, cap2);
        }
      // some token is not there, or after the tile's first row
      if (valid[0] != ~0u || (c + 1) * UNIT > lim_first) {
#pragma unroll
        for (int y = 0; y < NR; ++y)
#pragma unroll
          for (int x = 0; x < 2 * NS; ++x)
            if (!(valid[0] >> (nn + 8 * x) & 1) || c * UNIT + nn + 8 * x >= lim[y]) s[x][y] = -INFINITY;
      }
      float n[NR];
#pragma unroll
      for (int y = 0; y < NR; ++y) {
        n[y] = fmaxf(s[0][y], s[1][y]);
#pragma unroll
        for (int x = 2; x < 2 * NS; ++x) n[y] = fmaxf(n[y], s[x][y]);
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) n[y] = fmaxf(n[y], __shfl_xor_sync(0xffffffffu, n[y], x));
        n[y] = fmaxf(n[y], m[y]);
      }
      // the unit's largest |M|, of any group and token.  Those that are not finite do not count:
      // against them the other groups' would be zeros (their own products are NaN all the same)
      uint32_t bits = 0, vm[W];
      token_scales(here + at_vs + (lane & (UNIT - 1)) * scale_size + at_scales, vm);
#pragma unroll
      for (int g = 0; g < W; ++g) bits = __vmaxu2(bits, vm[g] & 0x7fff7fffu);
      bits = __reduce_max_sync(0xffffffffu, max(bits & 0xffffu, bits >> 16));
      if (bits >= kNotFinite) {
        bits = 0;
#pragma unroll
        for (int g = 0; g < W; ++g) {
          const uint32_t lo = vm[g] & 0x7fffu, hi = vm[g] >> 16 & 0x7fffu;
          bits = max(bits, max(lo < kNotFinite ? lo : 0u, hi < kNotFinite ? hi : 0u));
        }
        bits = __reduce_max_sync(0xffffffffu, bits);
      }
      const int e_new = max(top_m, Elem<E>::kBf16 ? (int)(bits >> 7) - 126 : (int)(bits >> 10) - 14);
      bool grown = e_new != top_m;
#pragma unroll
      for (int y = 0; y < NR; ++y) grown |= n[y] != m[y];
      if (__any_sync(0xffffffffu, grown)) {
        const float down = ex2((float)(top_m - e_new));
        top_m = e_new;
#pragma unroll
        for (int y = 0; y < NR; ++y) {
          const float fl = n[y] == m[y] ? 1.f : ex2(m[y] - n[y]), fo = fl * down;
          m[y] = n[y];
          l[y] *= fl;
#pragma unroll
          for (int g = 0; g < NO; ++g) {
            lg[g][y] *= fo;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[g][y][i] *= fo;
          }
        }
      }
      // ---- weights times 2^7, in one or two fp16 parts: both rows' or the one row's twice
      uint32_t ph[2 * NS], pl[2 * NS];
      float p[2 * NS][NR];
#pragma unroll
      for (int x = 0; x < 2 * NS; ++x) {
#pragma unroll
        for (int y = 0; y < NR; ++y) {
          // a row that has seen no key yet has m = -inf; its weights are zeros
          const float z = m[y] == -INFINITY ? 0.f : 7.f - m[y];
          p[x][y] = ex2(s[x][y] + z);
          l[y] += p[x][y];
        }
        ph[x] = Elem<__half>::from2(p[x][0], p[x][NR - 1]);
        if (kParts == 2) {
          const float2 h = Elem<__half>::to2(ph[x]);
          pl[x] = Elem<__half>::from2(p[x][0] - h.x, p[x][NR - 1] - h.y);
        }
      }
      // ---- the token's scales times 2^(7 - E) in fp16, and results
      const float m_up = __uint_as_float((uint32_t)(127 + 7 - top_m) << 23);
#pragma unroll
      for (int g = 0; g < W; ++g) {
        const float2 M = Elem<E>::to2(vm[g]);
        vm[g] = Elem<__half>::from2(M.x * m_up, M.y * m_up);
      }
      __syncwarp();                // (the last unit's are read)
      sts<W>(my_scales + (lane & (UNIT - 1)) * 2 * NG, vm);
      __syncwarp();
      uint32_t vf[4 * NS][W];
#pragma unroll
      for (int y = 0; y < 4 * NS; ++y) {
        const int t = (y >> 2) * 16 + 2 * kk + (y & 1) + (y & 2) * 4;
        if constexpr (FULL) {
          lds<W>(my_v + R::v_piece(t, nn * NG / 8) + nn * 2 * NG % 16, vf[y]);
        } else if constexpr (NC == 3) {                  // 6 bytes: two words, from the first's middle for odd nn
          uint32_t w0[1], w1[1];
          const int at = nn * 6 & ~3;
          lds<1>(my_v + R::v_piece(t, at >> 4) + (at & 15), w0);
          lds<1>(my_v + R::v_piece(t, (at + 4) >> 4) + ((at + 4) & 15), w1);
          vf[y][0] = nn & 1 ? w0[0] >> 16 | w1[0] << 16 : w0[0];
          vf[y][1] = nn & 1 ? w1[0] >> 16 : w1[0];
        } else {
#pragma unroll
          for (int g = 0; g < NC; ++g) {
            const int at = (nn * NC + g) * 2;
            const uint32_t h = lds_half(my_v + R::v_piece(t, at >> 4) + (at & 15));
            vf[y][g / 2] = g & 1 ? vf[y][g / 2] | h << 16 : h;
          }
        }
      }
#pragma unroll
      for (int ps = 0; ps < PASS; ++ps) {
        uint32_t bh[2 * NS], bl[2 * NS];
#pragma unroll
        for (int x = 0; x < 2 * NS; ++x) {
          // the scales of the lane's two columns
          uint32_t w1[1];
          lds<1>(my_scales + (nn + 8 * x) * 2 * NG + (RT == 8 ? ps / 2 : RT == 4 ? ps : 2 * ps + (kk & 1)) * 4, w1);
          const uint32_t w = RT == 8 ? __byte_perm(w1[0], w1[0], ps & 1 ? 0x3232 : 0x1010) : w1[0];
          const uint32_t hi = h2_mul(ph[x], w);
          // sums of p M: with one part of the product's own factors, as it has them, so that what
          // the codes' offset adds to a rounding cancels (an element that is zero stays zero); with two
          // of p and M themselves, from which the parts are 2^-21
          const float2 f = Elem<__half>::to2(kParts == 1 ? hi : w);
          auto sum = [&](float& to, float weight, float factor) { to = kParts == 1 ? to + factor : fmaf(weight, factor, to); };
          if constexpr (RT == 8) {
            sum(lg[ps][0], p[x][0], f.x);
            sum(lg[ps][NR - 1], p[x][NR - 1], kParts == 1 ? f.y : f.x);
          } else {
            sum(lg[2 * ps][0], p[x][0], f.x);
            if (2 * ps + 1 < NO) sum(lg[(2 * ps + 1) % NO][0], p[x][0], f.y);
          }
          bh[x] = trans8x8(hi);
          if (kParts == 2) bl[x] = trans8x8(h2_fma(pl[x], w, h2_fma(ph[x], w, h2_neg(hi))));
        }
        float acc[GC][2][4];
#pragma unroll
        for (int gi = 0; gi < GC; ++gi) {
          const int g = ps * GC + gi;
          if (g >= NC) {
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[gi][i >> 2][i & 3] = 0.f;
            continue;
          }
#pragma unroll
          for (int s2 = 0; s2 < NS; ++s2) {
            const uint32_t sel = g & 1 ? 0x7632 : 0x5410;
            const uint32_t ta = __byte_perm(vf[4 * s2][g / 2], vf[4 * s2 + 1][g / 2], sel);
            const uint32_t tb = __byte_perm(vf[4 * s2 + 2][g / 2], vf[4 * s2 + 3][g / 2], sel);
            const uint32_t ua = ta >> 8, ub = tb >> 8;
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
              const uint32_t b0 = part ? bl[2 * s2] : bh[2 * s2], b1 = part ? bl[2 * s2 + 1] : bh[2 * s2 + 1];
              if (s2 == 0 && part == 0) {
                mma_h(acc[gi][0], ta & kLow, ua & kLow, tb & kLow, ub & kLow, b0, b1, 0.f, 0.f, 0.f, 0.f);
                mma_h(acc[gi][1], ta & kHigh, ua & kHigh, tb & kHigh, ub & kHigh, b0, b1, 0.f, 0.f, 0.f, 0.f);
              } else {
                float(&c0)[4] = acc[gi][0], (&c1)[4] = acc[gi][1];
                mma_h(c0, ta & kLow, ua & kLow, tb & kLow, ub & kLow, b0, b1, c0[0], c0[1], c0[2], c0[3]);
                mma_h(c1, ta & kHigh, ua & kHigh, tb & kHigh, ub & kHigh, b0, b1, c1[0], c1[1], c1[2], c1[3]);
              }
            }
          }
          // element i of the lane's four: i / 2 the accumulator's row, i % 2 which of the two
          if constexpr (RT == 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int y = 0; y < 2; ++y) o[g][y % NR][i] += acc[gi][i & 1][(i & 2) + y];
          } else if constexpr (RT == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[g][0][i] += acc[gi][i & 1][(i & 2) + (g & 1)];
          }
        }
        if constexpr (RT == 2) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[2 * ps + j][0][i] += kk & 1 ? acc[2 % GC + j][i & 1][(i & 2) + j] : acc[j % GC][i & 1][(i & 2) + j];
        }
      }
#pragma unroll
      for (int x = 0; x < kAhead; ++x) valid[x] = valid[x + 1];
      stage = stage == R::kStages - 1 ? 0 : stage + 1;
    }
#pragma unroll
    for (int y = 0; y < NR; ++y) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[y] += __shfl_xor_sync(0xffffffffu, l[y], x);
#pragma unroll
      for (int g = 0; g < NO; ++g)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) lg[g][y] += __shfl_xor_sync(0xffffffffu, lg[g][y], x);
    }
    const bool whole = c0 == 0 && c1 == nchunk;
    const float m_down = __uint_as_float((uint32_t)(127 - 10 + top_m) << 23);     // 2^(E - 7) / 8
#pragma unroll
    for (int y = 0; y < NR; ++y) {
      const int row = my_row + y;
      if (row >= rows) continue;
      const float inv = l[y] == 0.f ? 0.f : 1.f / l[y];
      uint16_t* dst = a.out + (int64_t)dbg_index(q0 + row / group, a.T, d.error) * a.ldo +
                      (int64_t)(hk * group + row % group) * dim;
      // slot 0: the segment began in an earlier run; slot 1: it begins here
      const int64_t part = (((int64_t)grp * hbw + hsub) * 2 + (c0 == 0 ? 1 : 0)) * kKvRowTile + row - rt * RT;
#pragma unroll
      for (int gi = 0; gi < NO; ++gi) {
        const int g = RT == 2 ? gi / 2 * 4 + 2 * (kk & 1) + gi % 2 : gi, e = 32 * g + 4 * nn;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = fmaf(o[gi][y][i], i & 1 ? 0x1p20f : 0x1p24f, -7.f * lg[gi][y]) * inv * m_down;
        if (whole) {
          if (e < dim)
            *reinterpret_cast<uint2*>(dst + e) = make_uint2(Elem<E>::from2(v[0], v[1]), Elem<E>::from2(v[2], v[3]));
        } else {
          *reinterpret_cast<float4*>(a.part_o + part * (32 * NG) + e) = make_float4(v[0], v[1], v[2], v[3]);
        }
      }
      if (!whole && nn == 0 && (RT != 2 || (kk & 1) == 0)) a.part_ml[part] = make_float2(m[y], l[y]);
    }
    left -= c1 - c0;
    c0 = 0;                        // the next segment, if any is left
    if (++rt == tiles) {
      rt = 0;
      if (++hb == blocks) {
        hb = 0;
        ++r;
      }
    }
  }
  cp_wait<0>();
  if (missing) report_err(d.error, kErrInvalid);
  // after chunks: their kernel may still run, and this grid ends after it
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <class E, int NC, int RT>
cudaError_t launch_rows(KvAttendArgs a, int num_sms, bool after_chunks, cudaStream_t st) {
  constexpr int NG = q4_rounded(NC);
  // Heads of a CTA, and as many neighbouring ones at a time as up to 16 that several CTAs share:
  // a head's codes of a token are 64 bytes, and what neighbours read at other times the DRAM
  // fetches again (32 heads of 128, 256 requests: 121 us with a CTA's heads alone, 115 so; 8 key
  // heads, 128 long requests: 168 and 165).
  int heads = kMaxAbreast;
  while (a.kv.heads_kv % heads) --heads;
  a.hbw = std::max(1, 16 / heads) * heads;
  while (a.kv.heads_kv % a.hbw) a.hbw -= heads;
  static_assert(q4_warps(NC) <= kKvDecodeWarps, "the scratch has room for every warp's parts");
  const int grid = num_sms * (q4_warps(NC) / heads), smem = ring_bytes<NG>(heads, NC);
  const int threads = heads * 32;
  auto kernel = a.softcap > 0.f ? kv_q4_decode_kernel<E, NC, RT, true> : kv_q4_decode_kernel<E, NC, RT, false>;
  cudaError_t e;
  if (after_chunks) {
    e = launch_early(kernel, dim3(grid), threads, smem, st, a);
  } else {
    kernel<<<grid, threads, smem, st>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  return launch_kv_q4_join(a, Elem<E>::kBf16 ? 1 : 0, num_sms, after_chunks, grid / (a.hbw / heads), st);
}
template <class E, int NC, int RT>
cudaError_t prepare_rows() {
  for (auto k : {kv_q4_decode_kernel<E, NC, RT, false>, kv_q4_decode_kernel<E, NC, RT, true>})
    if (cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             ring_bytes<q4_rounded(NC)>(kMaxAbreast, NC) + 1024))
      return e;
  return cudaSuccess;
}
// What there is for a number of groups and a row tile (kv_q4_row_tile).
template <class E>
struct Rows {
  cudaError_t (*launch)(KvAttendArgs, int, bool, cudaStream_t);
  cudaError_t (*prepare)();
  template <int NC, int RT>
  static constexpr Rows of() { return {launch_rows<E, NC, RT>, prepare_rows<E, NC, RT>}; }
  static Rows get(int groups, int tile) {
    switch (groups * 16 + tile) {
      case 2 * 16 + 4: return of<2, 4>();
      case 2 * 16 + 8: return of<2, 8>();
      case 3 * 16 + 2: return of<3, 2>();
      case 3 * 16 + 4: return of<3, 4>();
      case 3 * 16 + 8: return of<3, 8>();
      case 4 * 16 + 2: return of<4, 2>();
      case 4 * 16 + 4: return of<4, 4>();
      case 4 * 16 + 8: return of<4, 8>();
      case 5 * 16 + 2: return of<5, 2>();
      case 5 * 16 + 8: return of<5, 8>();
      case 6 * 16 + 2: return of<6, 2>();
      case 6 * 16 + 8: return of<6, 8>();
      case 7 * 16 + 2: return of<7, 2>();
      case 7 * 16 + 8: return of<7, 8>();
      case 8 * 16 + 2: return of<8, 2>();
      case 8 * 16 + 8: return of<8, 8>();
      default: return of<1, 8>();
    }
  }
};
template <class E>
cudaError_t prepare_all(int groups) {
  for (int tile : {2, 4, 8})
    if (cudaError_t e = Rows<E>::get(groups, tile).prepare()) return e;
  return cudaSuccess;
}

}  // namespace

cudaError_t prepare_kv_q4_decode_kernels(int dtype, int groups) {
  return dtype == 0 ? prepare_all<__half>(groups) : prepare_all<__nv_bfloat16>(groups);
}

cudaError_t launch_kv_q4_decode(const KvAttendArgs& a, int dtype, int num_sms, bool after_chunks, cudaStream_t st) {
  return dtype == 0 ? Rows<__half>::get(a.kv.groups, a.row_tile).launch(a, num_sms, after_chunks, st)
                    : Rows<__nv_bfloat16>::get(a.kv.groups, a.row_tile).launch(a, num_sms, after_chunks, st);
}

}  // namespace slora
