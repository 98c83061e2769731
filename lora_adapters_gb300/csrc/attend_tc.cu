// slora_kv_attend for chunks: many new tokens of one request over its paged
// keys and values, on the tensor cores (tcgen05).
//
// Rows are (token, query head) pairs that share a key head: a tile of 128 of
// them is 128 / group tokens of the request with all `group` heads each, so
// shared key heads fill the tile as well as separate ones do.  Per 128 keys
//     S = Q K^T        (128 x 128 x head_dim, operands in shared memory)
//     P = 2^(scale' S - m), m the row's running maximum in powers of two
//     O <- O 2^(m_old - m) + P V       (P from TMEM, V in shared memory)
// and O / sum(P) at the end.  S, P and O live in TMEM; S is read once and P,
// rounded to the storage type (its sum is taken before the rounding), written
// over it.  The rounding adds at most one unit of the storage type relative to
// the largest value, the size of the result's own rounding.  fp16 has few
// exponents, so there P is 2^7 times that (its sum alike, which the quotient
// undoes): 11 bits for weights above 2^-21 of 2^m, an error of 2^-32 of it below,
// and at most 2^15 where the maximum has grown past m.
//
// Bound: the tensor cores where contexts are long (4 head_dim operations per
// score against a softmax of about ten instructions, the exponentials first),
// memory for prompts of a few hundred tokens.  What the layout is for:
//  - two tiles (A, B) of one request and key head share every K and V tile and
//    take turns: while one tile's softmax runs, the tensor cores work on the
//    other's products;
//  - O is rescaled only when a row's maximum has grown by more than 2^8 (e^(s - m)
//    then stays below 2^8, and fp32 sums lose nothing by it);
//  - keys and values are gathered from their pages by four warps with 16-byte
//    asynchronous copies into a ring of tiles;
//  - the work, (request, key head, pair of tiles) x 128-key tiles laid end to
//    end, is cut into equal runs, one per CTA; what a run holds of a segment
//    cut by its ends goes to scratch as (m, l, O), joined in order afterwards.
// A position past the request's length, or one whose table entry names no page,
// reads nothing: its key and value are zeros and its weight is 0.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "kv.cuh"
#include "kv.h"
#include "ptx.cuh"

namespace slora {
namespace {

using namespace ptx;

constexpr int kRowBytes = 128;                  // 64 elements, one swizzle row
constexpr int kAtom = kKvTile * kRowBytes;      // 128 rows x 64 elements: 16 KB
constexpr int kMaxAtoms = 2;                    // head_dim <= 128
constexpr int kStages = 4;                      // K and V tiles in flight
constexpr int kQTiles = 3;                      // Q tiles: two in use, one for the next part
// warps: 0-3 K and V, 4-7 softmax of tile A, 8-11 of tile B, 12 MMAs, 13 Q,
// 14 the walk
constexpr int kThreads = 16 * 32;
constexpr int kLoaders = 4 * 32;
constexpr int kWarpMma = 12, kWarpQ = 13, kWarpWalk = 14;
constexpr int kParts = 4;                       // parts handed out ahead
constexpr int kPartReaders = 4 + 8 + 2;         // warps that read them
// Registers a thread of each warp group (setmaxnreg): the launch gives each of
// the four groups 128, and the shares add up to the same 512.
constexpr int kRegsLoad = 48, kRegsSoftmax = 192, kRegsOther = 80;
static_assert(kRegsLoad + 2 * kRegsSoftmax + kRegsOther <= 4 * 128, "the shares come out of the launch's registers");
constexpr int kTmemCols = 512;                  // S_A, S_B, O_A, O_B of 128 columns each
constexpr float kGrow = 8.f;                    // O is rescaled when a maximum grew by more (powers of two)

// A wait gives up after kWaitLimit polls (SLORA_ERR_TIMEOUT).  The longest
// honest one is the query loader's, for a part of the run: 40 ms for the
// largest cache that fits this GPU.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitLimit; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Pairs of fp32 in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Matrix descriptors as their low words (start address and leading offset in
// 16-byte units): the high word, stride offset 1024 and 128-byte swizzle, is
// the same for all of them.
constexpr uint32_t kDescHi = (uint32_t)((uint64_t)(1024 >> 4) | (1u << 14) | (2u << 29));
__device__ __forceinline__ uint32_t desc_lo(const void* p, uint32_t lbo_bytes) {
  return ((smem_addr(p) >> 4) & 0x3FFFu) | ((lbo_bytes >> 4) << 16);
}
// D[tmem] (+)= A[smem] B[smem].
template <bool ADD>
__device__ __forceinline__ void umma_ss(uint32_t tmem_d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
      "setp.ne.b32 p, %5, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(kDescHi), "n"(ADD ? 1 : 0));
}
// D[tmem] (+)= A[tmem] B[smem]: A is 128 lanes of packed 16-bit pairs.
__device__ __forceinline__ void umma_ts(uint32_t tmem_d, uint32_t tmem_a, uint32_t b_lo, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %4};\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "r"(b_lo), "r"(idesc), "n"(kDescHi), "r"(add));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}
// 16 bytes global -> shared, not kept in L1; bytes = 0: zeros, nothing is read.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// One arrival on the barrier when all copies of this thread so far have landed.
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// True in one lane of a converged warp, always the same one.  The MMA role runs
// in that lane alone, waits and all: with the whole warp in the loop and one
// lane of it issuing, every step took four times as long (741 us instead of
// 319 for a 1024-token chunk over 16 K tokens).
__device__ __forceinline__ bool elect_one() {
  uint32_t y;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(y));
  return y != 0;
}
// 3-D tiled tensor copy global -> shared.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// S = Q K^T of STEPS 16-element steps; q, k: descriptors of the tiles.
template <int STEPS>
__device__ __forceinline__ void issue_qk(uint32_t tmem_s, uint32_t q, uint32_t k, uint32_t idesc) {
  umma_ss<false>(tmem_s, q, k, idesc);
#pragma unroll
  for (int ks = 1; ks < STEPS; ++ks) {
    const uint32_t o = (ks >> 2) * (kAtom / 16) + (ks & 3) * 2;
    umma_ss<true>(tmem_s, q + o, k + o, idesc);
  }
}

// A part of a segment: one request, key head and pair of tiles, key tiles
// [i0, i1) of n.  One warp walks the CTA's run and hands the parts to the other
// roles through shared memory, a few ahead.
struct alignas(16) Part {
  int i0, i1;              // key tiles of this part (i1 = 0: the run is over)
  int end[2];              // one past the last key tile that tile A (B) of the pair needs, i0: none
  int tok, pos, tokens[2]; // the pair's first token and its position; tokens of tile A, of tile B
  int hk, row, len, whole; // key head; table row; tokens held; the segment lies in this part as a whole
  int last, pad[3];        // the CTA whose run ends the segment
};
static_assert(sizeof(Part) == 64, "four 16-byte pieces");
// Walks a CTA's run of units part by part.
// A pair of tiles with n key tiles is kKvPairUnits + n units, the first ones its
// own cost; a run that ends within those leaves the pair to the next CTA.
struct Walk {
  int64_t u;               // the next part's first unit
  int left;                // units of the run not yet walked
  int r, hk, pr, v0;       // where the next part starts: request, key head, pair, unit of the pair
};
// Key tiles of pair pr: up to the position of its last token.
__device__ __forceinline__ int pair_tiles(int ctx, int fresh, int tpt, int pr) {
  return (ctx + min(fresh, (pr + 1) * 2 * tpt) + kKvTile - 1) / kKvTile;
}
// The walk from unit u on.
__device__ __forceinline__ Walk walk_start(const KvAttendArgs& a, int64_t u, int64_t end) {
  const KvDev& d = a.kv;
  int lo = 0, hi = a.R - 1;         // the last request that starts at or before u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int64_t)__ldg(d.tc_off + mid) * d.heads_kv <= u) lo = mid;
    else hi = mid - 1;
  }
  const int off = __ldg(d.tc_off + lo), per = max(1, __ldg(d.tc_off + lo + 1) - off);
  const int64_t in = u - (int64_t)off * d.heads_kv;
  Walk w;
  w.u = u;
  w.left = (int)(end - u);
  w.r = lo;
  w.hk = (int)(in / per);
  w.v0 = (int)(in - (int64_t)w.hk * per);
  w.pr = 0;
  const int4 rq = __ldg(d.req + lo);
  const int fresh = rq.y, ctx = rq.z - fresh;
  for (int n; w.v0 >= (n = kKvPairUnits + pair_tiles(ctx, fresh, a.tpt, w.pr)); ++w.pr) w.v0 -= n;
  return w;
}
__device__ __forceinline__ Part walk_next(const KvAttendArgs& a, Walk& w, int64_t run) {
  Part p{};
  const KvDev& d = a.kv;
  while (w.left > 0 && p.i1 == 0) {
    const int4 rq = __ldg(d.req + w.r);
    const int q0 = rq.x, fresh = rq.y;
    p.len = rq.z;
    p.row = rq.w;
    const int ctx = p.len - fresh, t0 = w.pr * 2 * a.tpt, n = pair_tiles(ctx, fresh, a.tpt, w.pr);
    const int v1 = min(kKvPairUnits + n, w.v0 + w.left);
    p.i0 = max(0, w.v0 - kKvPairUnits);
    p.i1 = max(0, v1 - kKvPairUnits);
    p.tok = q0 + t0;
    p.pos = ctx + t0;
    p.hk = w.hk;
    p.whole = p.i0 == 0 && p.i1 == n;
    p.last = (int)((w.u - w.v0 + kKvPairUnits + n - 1) / run);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      p.tokens[x] = max(0, min(a.tpt, fresh - t0 - x * a.tpt));
      p.end[x] = p.tokens[x] == 0 ? p.i0
                                  : max(p.i0, min(p.i1, (p.pos + x * a.tpt + p.tokens[x] + kKvTile - 1) / kKvTile));
    }
    w.left -= v1 - w.v0;
    w.u += v1 - w.v0;
    w.v0 = 0;
    if (w.left > 0) {                 // the next pair, key head or request with tiles
      if (++w.pr * 2 * a.tpt >= fresh) {
        w.pr = 0;
        if (++w.hk == d.heads_kv) {
          w.hk = 0;
          do ++w.r;
          while (__ldg(d.tc_off + w.r + 1) == __ldg(d.tc_off + w.r));
        }
      }
    }
  }
  return p;
}

struct TcSmem {
  uint8_t q[kQTiles][kMaxAtoms][kAtom];
  uint8_t kv[kStages][kMaxAtoms][kAtom];
  uint64_t q_full[kQTiles], q_empty[kQTiles], kv_full[kStages], kv_empty[kStages];
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
  uint64_t part_full[kParts], part_empty[kParts];
  Part part[kParts];
  // Positions of a K tile whose entry names no page, a bit each, in the word of the
  // warp that loads them.  Tile k is loaded when the scores of tile k - 2 are done,
  // which begin after the softmax of tile k - 3: of four places, k - 4's is free.
  alignas(16) uint32_t holes[4][4];
  uint32_t tmem_slot;
};

// STEPS: 16-element steps of a head, 8 or 4; 0: head_dim 80, 96 or 112 (a
// branch to the right run of MMAs costs 7 % of the kernel).
// CAP: scores as they are, capped with softcap <= kCapNear, or with any softcap (a
// 1024-token chunk over 16 K tokens, 40 query heads on 8: 263, 486 and 747 us).
enum { kCapNone = 0, kCapSmall, kCapAny };
template <class E, int CAP, int STEPS>
__global__ void __launch_bounds__(kThreads, 1) kv_chunk_kernel(const __grid_constant__ KvAttendArgs a) {
  extern __shared__ uint8_t smem_raw[];
  TcSmem& sm = *reinterpret_cast<TcSmem*>(smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023));
  const KvDev& d = a.kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t total = (int64_t)__ldg(d.tc_off + a.R) * d.heads_kv;
  const int64_t run = (total + gridDim.x - 1) / gridDim.x;
  pdl_trigger();        // the decode kernel's CTAs take the SMs that become free
  if ((int64_t)blockIdx.x * run >= total) {
    if (threadIdx.x == 0) a.tc_split[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  if (warp == kWarpMma) tmem_alloc(&sm.tmem_slot, kTmemCols);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.kv_full[s], kLoaders + (s & 1 ? 0 : 4));   // even stages hold K tiles, whose holes come with them
      mbar_init(&sm.kv_empty[s], 1);
    }
    for (int k = 0; k < kParts; ++k) {
      mbar_init(&sm.part_full[k], 1);
      mbar_init(&sm.part_empty[k], kPartReaders);
    }
    for (int b = 0; b < kQTiles; ++b) {
      mbar_init(&sm.q_full[b], 1);
      mbar_init(&sm.q_empty[b], 4);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sm.s_full[x], 1);
      mbar_init(&sm.p_full[x], 4);
      mbar_init(&sm.o_full[x], 1);
      mbar_init(&sm.o_empty[x], 4);
    }
    mbar_fence_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_slot;
  const int dim = d.head_dim, group = d.heads_q / d.heads_kv, tpt = a.tpt;
  const int natoms = (dim + 63) >> 6;
  bool ok = true;
  // by a whole warp: every lane polls (one lane polling and a shuffle that
  // tells the others cost 6 % of the kernel)
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait_bar(bar, parity));
  };
  // the reader's next part (false: no more, or a wait gave up): copied out of
  // the ring by every lane, handed back by one
  uint32_t n_part = 0;
  auto next_part = [&](Part& p, bool whole_warp) -> bool {
    const uint32_t k = n_part % kParts, ph = (n_part / kParts) & 1;
    if (!ok || !(whole_warp ? wait_warp(&sm.part_full[k], ph) : wait_bar(&sm.part_full[k], ph))) {
      ok = false;
      return false;
    }
    ++n_part;
    p = sm.part[k];
    return true;
  };
  auto part_read = [&]() { mbar_arrive(&sm.part_empty[(n_part - 1) % kParts]); };
  Part p;

  if (warp < 4) {  // -------------------------------------------------- K and V tiles
    // Warp w copies rows 32 w .. 32 w + 31 of a tile, a lane 16 bytes of every
    // fourth row, straight to their swizzled places; each lane looks one
    // position's page up, for the next tile while this one's copies run.  The
    // copies arrive on the tile's barrier when they land, so a warp runs the
    // whole ring ahead.
    regs_down<kRegsLoad>();
    const int64_t plane = (int64_t)d.max_rows * d.max_blocks;
    const int64_t row_bytes = (int64_t)d.heads_kv * dim * 2;
    const int ch = lane & 7, sub = lane >> 3;
    const bool ch1 = 64 + ch * 8 < dim;              // this lane's piece of the second atom exists
    uint32_t n = 0;      // tiles issued
    for (;;) {
      if (!next_part(p, true)) break;
      __syncwarp();
      if (lane == 0) part_read();
      if (p.i1 == 0) break;
      const int32_t* tab = d.table + 2 * a.layer * plane + (int64_t)dbg_index(p.row, d.max_rows, d.error) * d.max_blocks;
      const uint8_t* base = reinterpret_cast<const uint8_t*>(d.pool) + (int64_t)p.hk * dim * 2 + ch * 16;
      int kslot, vslot;            // pool rows, -1: none
      uint32_t holes;
      auto lookup = [&](int i) {
        const int j = i * kKvTile + 32 * warp + lane;
        kslot = vslot = -1;
        if (j < p.len) {
          const int b = (int)a.per_page_div.div((uint32_t)j), off = j - b * d.per_page;
          const int kp = __ldg(tab + b), vp = __ldg(tab + plane + b);
          if ((uint32_t)kp < (uint32_t)d.num_pages && (uint32_t)vp < (uint32_t)d.num_pages) {
            kslot = kp * d.per_page + off;
            vslot = vp * d.per_page + off;
          }
        }
        holes = __ballot_sync(0xffffffffu, j < p.len && kslot < 0);
        if (holes && lane == 0) report_err(d.error, kErrInvalid);
      };
      lookup(p.i0);
      for (int i = p.i0; i < p.i1 && ok; ++i) {
        const int kc = kslot, vc = vslot;
        const uint32_t hc = holes;
        if (i + 1 < p.i1) lookup(i + 1);
#pragma unroll
        for (int half = 0; half < 2; ++half, ++n) {
          const uint32_t st = n % kStages;
          if (!wait_warp(&sm.kv_empty[st], ((n / kStages) & 1) ^ 1)) {
            ok = false;
            break;
          }
          const uint32_t dst = smem_addr(sm.kv[st][0]) + (32 * warp + sub) * kRowBytes;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int row = __shfl_sync(0xffffffffu, half ? vc : kc, 4 * j + sub);
            const uint8_t* src = base + max(row, 0) * row_bytes;
            const uint32_t bytes = row < 0 ? 0 : 16;
            // row 32 w + 4 j + sub of the tile; its chunk ch goes to ch ^ (row & 7)
            const uint32_t to = dst + 4 * j * kRowBytes + ((ch ^ ((4 * j + sub) & 7)) << 4);
            cp16(to, src, bytes);
            if (ch1) cp16(to + kAtom, src + 128, bytes);
          }
          if (half == 0 && lane == 0) {
            sm.holes[(n >> 1) & 3][warp] = hc;
            mbar_arrive(&sm.kv_full[st]);
          }
          cp_arrive(&sm.kv_full[st]);
        }
      }
      if (!ok) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= 12) {
    regs_down<kRegsOther>();
    if (warp == kWarpQ) {  // ----------------------------------------------- Q tiles
      if (elect_one()) {
        uint32_t n = 0;      // tiles loaded
        while (next_part(p, false)) {
          part_read();
          if (p.i1 == 0) break;
          for (int x = 0; x < 2 && ok; ++x) {
            if (p.end[x] == p.i0) continue;      // no keys for this tile here
            const uint32_t b = n % kQTiles;
            ok = wait_bar(&sm.q_empty[b], ((n / kQTiles) & 1) ^ 1);
            if (!ok) break;
            mbar_expect_tx(&sm.q_full[b], (uint32_t)(natoms * tpt * group) * kRowBytes);
            for (int at = 0; at < natoms; ++at)
              tma_load_3d(sm.q[b][at], &a.q_map, at * 64, p.hk * group, p.tok + x * tpt, &sm.q_full[b]);
            ++n;
          }
        }
        for (uint32_t k = n > kQTiles ? n - kQTiles : 0; k < n; ++k)   // copies land before the CTA goes
          wait_bar(&sm.q_full[k % kQTiles], (k / kQTiles) & 1);
      }
    } else if (warp == kWarpWalk) {  // ------------------------------------- the walk, by one thread
      if (elect_one()) {
        const int64_t u0 = (int64_t)blockIdx.x * run;
        Walk w = walk_start(a, u0, min(total, u0 + run));
        int4 split = make_int4(-1, 0, 0, 0);
        for (uint32_t k = 0;; ++k) {
          const Part q = walk_next(a, w, run);
          if (q.i1 > 0 && q.i0 == 0 && !q.whole)      // a split segment begins here
            split = make_int4(q.tok, q.tokens[0] << 16 | q.tokens[1], q.hk, q.last);
          ok = wait_bar(&sm.part_empty[k % kParts], ((k / kParts) & 1) ^ 1);
          if (!ok) break;
          sm.part[k % kParts] = q;
          mbar_arrive(&sm.part_full[k % kParts]);
          if (q.i1 == 0) break;
        }
        a.tc_split[blockIdx.x] = split;
      }
    } else if (warp == kWarpMma && elect_one()) {  // ----------------------- MMAs, by one thread
      const uint32_t id_s = umma_idesc_f16(kKvTile, kKvTile, Elem<E>::kBf16, false);
      const uint32_t id_o = umma_idesc_f16(kKvTile, dim, Elem<E>::kBf16, true);
      // descriptors of the first tiles; others by adding to the address field
      // (16-byte units), one addition an instruction
      const uint32_t q_desc = desc_lo(sm.q[0][0], 16), k_desc = desc_lo(sm.kv[0][0], 16),
                     v_desc = desc_lo(sm.kv[0][0], kAtom);
      constexpr uint32_t kTileUnits = kMaxAtoms * kAtom / 16;
      uint32_t st = 0, ph = 0;                  // the ring's next tile
      uint32_t p_ph = 0, o_ph = 3;              // a bit per tile: the phase to wait for
      uint32_t nq = 0;                          // Q tiles used
      auto issue_s = [&](int x, uint32_t qb, uint32_t kst) {
        const uint32_t qd = q_desc + qb * kTileUnits, kd = k_desc + kst * kTileUnits;
        const uint32_t ts = tmem + x * 128;
        if constexpr (STEPS > 0) {
          issue_qk<STEPS>(ts, qd, kd, id_s);
        } else {
          switch (dim) {
            case 80: issue_qk<5>(ts, qd, kd, id_s); break;
            case 96: issue_qk<6>(ts, qd, kd, id_s); break;
            default: issue_qk<7>(ts, qd, kd, id_s); break;
          }
        }
        umma_commit(&sm.s_full[x]);
      };
      auto issue_o = [&](int x, uint32_t vst, uint32_t add) {
        const uint32_t vd = v_desc + vst * kTileUnits;
#pragma unroll
        for (int ks = 0; ks < kKvTile / 16; ++ks)
          umma_ts(tmem + 256 + x * 128, tmem + x * 128 + ks * 8, vd + ks * (16 * kRowBytes / 16), id_o, ks ? 1u : add);
      };
      while (next_part(p, false)) {
        part_read();
        if (p.i1 == 0) break;
        const int end0 = p.end[0], end1 = p.end[1];
        const uint32_t n0 = nq, n1 = nq + (end0 > p.i0);    // the tiles' places in the order of loads
        nq = n1 + (end1 > p.i0);
        const uint32_t qb0 = n0 % kQTiles, qb1 = n1 % kQTiles;
        // K tile i + 1 and V tile i, in the order they were loaded (K i0, V i0, K i0 + 1, ...)
        for (int i = p.i0 - 1; i < p.i1 && ok; ++i) {
          const bool has_v = i >= p.i0, has_k = i + 1 < p.i1;
          const uint32_t vst = st;
          if (has_v) {
            ok = wait_bar(&sm.kv_full[st], ph);
            if (++st == kStages) {
              st = 0;
              ph ^= 1;
            }
          }
          const uint32_t kst = st;
          // (a K tile that no tile needs is waited for all the same: its slot
          // may only be handed back once it has been filled)
          bool k_in = !has_k;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int end = x ? end1 : end0;
            if (ok && has_v && i < end) {
              if (i == p.i0) {        // O of the tile's previous part has been read
                ok = wait_bar(&sm.o_empty[x], (o_ph >> x) & 1);
                o_ph ^= 1u << x;
              }
              ok = ok && wait_bar(&sm.p_full[x], (p_ph >> x) & 1);
              tc_fence_after();
              fence_async_shared();   // the tile's copies (generic proxy), for the MMAs' reads
              p_ph ^= 1u << x;
              if (ok) {
                issue_o(x, vst, i > p.i0 ? 1u : 0u);
                if (i == end - 1) umma_commit(&sm.o_full[x]);
              }
            }
            if (ok && !k_in) {
              ok = wait_bar(&sm.kv_full[kst], ph);
              k_in = true;
              tc_fence_after();
              fence_async_shared();
            }
            if (ok && i + 1 < end) {
              if (!has_v) {             // the part's first: this tile's queries
                ok = wait_bar(&sm.q_full[x ? qb1 : qb0], ((x ? n1 : n0) / kQTiles) & 1);
              }
              if (ok) issue_s(x, x ? qb1 : qb0, kst);
            }
          }
          if (!ok) break;
          if (has_v) umma_commit(&sm.kv_empty[vst]);
          if (has_k) umma_commit(&sm.kv_empty[kst]);
          if (has_k && ++st == kStages) {
            st = 0;
            ph ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else {  // --------------------------------------------------------- softmax
    regs_up<kRegsSoftmax>();
    const int x = (warp - 4) >> 2, quarter = warp & 3, rho = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t t_s = tmem + lanes + x * 128, t_o = tmem + lanes + 256 + x * 128;
    const float sc = kLog2e * a.scale, cap_t = a.cap_t, cap2 = a.cap2;
    constexpr float kUp = Elem<E>::kBf16 ? 0.f : 7.f;        // weights are held times 2^kUp
    const int my_tok = rho / group, my_head = rho - my_tok * group;
    uint32_t ns = 0, nf = 0, nq = 0, nk = 0;                  // nk: K tiles of earlier parts
    for (;;) {
      if (!next_part(p, true)) break;
      __syncwarp();
      if (lane == 0) part_read();
      if (p.i1 == 0) break;
      const int end = x ? p.end[1] : p.end[0], tokens = x ? p.tokens[1] : p.tokens[0];
      const uint32_t has0 = p.end[0] > p.i0, has1 = p.end[1] > p.i0, qb = (nq + (x ? has0 : 0)) % kQTiles;
      nq += has0 + has1;
      const uint32_t k0 = nk - p.i0;
      nk += p.i1 - p.i0;
      const bool live = my_tok < tokens;
      const int pos_first = p.pos + x * tpt;                  // the tile's earliest position
      const int pos = pos_first + min(my_tok, max(tokens - 1, 0));
      float m = -INFINITY;
      float l = 0.f;
      for (int i = p.i0; i < end; ++i) {
        if (!wait_warp(&sm.s_full[x], ns & 1)) {
          ok = false;
          break;
        }
        ++ns;
        tc_fence_after();
        // S, 32 columns at a time: the next ones on their way while these are
        // capped, masked and searched for the maximum
        uint32_t s[4][32];
        const int lim = pos - i * kKvTile;
        float mx = -INFINITY, my = -INFINITY;
        tmem_ld32_nowait(t_s, s[0]);
        const uint4 hole = *reinterpret_cast<const uint4*>(sm.holes[(k0 + i) & 3]);
        // some row may not see the whole tile
        const bool edge = (i + 1) * kKvTile - 1 > pos_first || (hole.x | hole.y | hole.z | hole.w) != 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_wait_ld(s[c]);
          if (c < 3) tmem_ld32_nowait(t_s + 32 * (c + 1), s[c + 1]);
          if (CAP) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              s[c][j] = __float_as_uint(capped<CAP == kCapAny>(__uint_as_float(s[c][j]), sc, cap_t, cap2));
          }
          if (edge) {
            const uint32_t gone = (lim >= 32 * c + 31 ? 0u : lim < 32 * c ? ~0u : ~1u << (lim - 32 * c)) |
                                  (c == 0 ? hole.x : c == 1 ? hole.y : c == 2 ? hole.z : hole.w);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if ((gone >> j) & 1) s[c][j] = 0xff800000u;     // -inf
          }
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            mx = max3(mx, __uint_as_float(s[c][j]), __uint_as_float(s[c][j + 1]));
            my = max3(my, __uint_as_float(s[c][j + 2]), __uint_as_float(s[c][j + 3]));
          }
        }
        mx = fmaxf(mx, my);
        if (!CAP) mx *= sc;                                   // scale > 0; -inf stays
        if (i == p.i0) {
          m = mx;
        } else if (__any_sync(0xffffffffu, live && (mx > m + kGrow || (m == -INFINITY && mx > m)))) {
          // the products up to the previous tile are done (S came after them).
          // Rows without a query have no vote: they hold what an earlier part
          // left, and when the others are rescaled shows in their last bits.
          const float mn = fmaxf(m, mx);
          const float f = mn == m ? 1.f : ex2(m - mn);
          m = mn;
          l *= f;
#pragma unroll 1
          for (int c = 0; c < dim; c += 16) {
            float v[16];
            uint32_t r[16];
            tmem_ld16(t_o + c, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(v[j] * f);
            tmem_st16(t_o + c, r);
          }
        }
        const float z = m == -INFINITY ? 0.f : m - kUp;       // a row that sees nothing yet: all weights 0
        // a tile's weights are added up first: one by one, small ones are lost beside a large sum
        uint64_t l2a = 0, l2b = 0;                            // pairs of partial sums (+0, +0)
        const uint64_t sc2 = CAP ? pair(1.f, 1.f) : pair(sc, sc), z2 = pair(-z, -z);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float2 e0 = unpair(fma2(pair(__uint_as_float(s[c][j]), __uint_as_float(s[c][j + 1])), sc2, z2));
            const float2 e1 = unpair(fma2(pair(__uint_as_float(s[c][j + 2]), __uint_as_float(s[c][j + 3])), sc2, z2));
            const float p0 = ex2(e0.x), p1 = ex2(e0.y), p2 = ex2(e1.x), p3 = ex2(e1.y);
            l2a = add2(l2a, pair(p0, p1));
            l2b = add2(l2b, pair(p2, p3));
            pk[j / 2] = Elem<E>::from2(p0, p1);
            pk[j / 2 + 1] = Elem<E>::from2(p2, p3);
          }
          tmem_st16(t_s + 16 * c, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[x]);
        const float2 la = unpair(l2a), lb = unpair(l2b);
        l += (la.x + la.y) + (lb.x + lb.y);
      }
      if (!ok) break;
      const bool whole = p.whole != 0;
      // slot 0: the segment began in an earlier run; slot 1: it begins here
      const int64_t part = (((int64_t)blockIdx.x * 2 + (p.i0 == 0 ? 1 : 0)) * 2 + x) * kKvTile + rho;
      if (end > p.i0) {
        if (!wait_warp(&sm.o_full[x], nf & 1)) {
          ok = false;
          break;
        }
        ++nf;
        tc_fence_after();
        // The tile's rows leave through its queries' place in shared memory
        // (their last product is done), 256 bytes a row in 16-byte pieces, the
        // piece's place exchanged by the row's low bits: each warp writes its
        // own 32 rows one row a lane and reads them back row by row, so that
        // global memory sees whole rows.
        uint8_t* stage = sm.q[qb][0] + 32 * quarter * 256;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int tok = p.tok + x * tpt + my_tok;
        uint8_t* dst = whole ? reinterpret_cast<uint8_t*>(a.out + (int64_t)(live ? dbg_index(tok, a.T, d.error) : tok) * a.ldo +
                                                          (int64_t)(p.hk * group + my_head) * dim)
                             : reinterpret_cast<uint8_t*>(a.tc_part_o + part * kKvTile);
        const uint32_t rows_live = __ballot_sync(0xffffffffu, live);
        const int piece = lane & 15;
        uint8_t* mine = stage + lane * 256;
        // (loops kept rolled: code run once per part is fetched as it runs)
        auto store_rows = [&](int byte0, int bytes) {
          __syncwarp();
#pragma unroll 1
          for (int r0 = lane >> 4; r0 < 32; r0 += 8) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int rr = r0 + 2 * k;
              v[k] = *reinterpret_cast<const uint4*>(stage + rr * 256 + (piece ^ (rr & 7)) * 16);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int rr = r0 + 2 * k;
              uint8_t* to = reinterpret_cast<uint8_t*>(
                  __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), rr));
              if (((rows_live >> rr) & 1) && piece * 16 < bytes) *reinterpret_cast<uint4*>(to + byte0 + piece * 16) = v[k];
            }
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {      // 32 columns (beyond head_dim: whatever is there, not stored)
          uint32_t o[32];
          tmem_ld32_nowait(t_o + 32 * c, o);
          tmem_wait_ld(o);
          if (whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float y[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) y[j] = __uint_as_float(o[k * 8 + j]) * inv;
              *reinterpret_cast<uint4*>(mine + ((4 * c + k) ^ (lane & 7)) * 16) = pack8<E>(y);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(mine + ((8 * (c & 1) + k) ^ (lane & 7)) * 16) =
                  make_uint4(o[k * 4], o[k * 4 + 1], o[k * 4 + 2], o[k * 4 + 3]);
            if (c & 1) store_rows(128 * (c - 1), dim * 4 - 128 * (c - 1));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_empty[x]);        // the next part's products may start
        if (whole) store_rows(0, dim * 2);
        fence_async_shared();      // the next queries come through the TMA engine
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_empty[qb]);
      }
      if (!whole && live) a.tc_part_ml[part] = make_float2(m, l);   // l = 0: the part has no weight, O unwritten
    }
  }
  if (!ok) report_err(d.error, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

constexpr size_t kSmemBytes = sizeof(TcSmem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");

template <class E, int CAP>
void (*chunk_kernel(int head_dim))(const KvAttendArgs) {
  return head_dim == 128 ? kv_chunk_kernel<E, CAP, 8> : head_dim == 64 ? kv_chunk_kernel<E, CAP, 4>
                                                                       : kv_chunk_kernel<E, CAP, 0>;
}
template <class E>
void (*chunk_kernel(int cap, int head_dim))(const KvAttendArgs) {
  return cap == kCapNone ? chunk_kernel<E, kCapNone>(head_dim)
                         : cap == kCapSmall ? chunk_kernel<E, kCapSmall>(head_dim) : chunk_kernel<E, kCapAny>(head_dim);
}
void (*chunk_kernel(int dtype, int cap, int head_dim))(const KvAttendArgs) {
  return dtype == 0 ? chunk_kernel<__half>(cap, head_dim) : chunk_kernel<__nv_bfloat16>(cap, head_dim);
}

}  // namespace

cudaError_t prepare_kv_chunk_kernels() {
  for (int dtype = 0; dtype < 2; ++dtype)
    for (int cap : {kCapNone, kCapSmall, kCapAny})
      for (int head_dim : {64, 80, 128}) {
        const cudaError_t e = cudaFuncSetAttribute(chunk_kernel(dtype, cap, head_dim),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

int64_t kv_chunk_part_rows(int num_sms) { return (int64_t)num_sms * 4 * kKvTile; }

cudaError_t launch_kv_chunk(const KvAttendArgs& a, int dtype, int num_sms, cudaStream_t st) {
  const int cap = a.softcap == 0.f ? kCapNone : a.softcap <= kCapNear ? kCapSmall : kCapAny;
  chunk_kernel(dtype, cap, a.kv.head_dim)<<<num_sms, kThreads, kSmemBytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace slora
