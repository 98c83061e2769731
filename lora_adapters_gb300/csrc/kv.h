// Internal interface of the paged key-value cache: kv.cpp (host), kv.cu, kv_q4.cu,
// attend.cu, attend_tc.cu and attend_q4.cu (kernels), pool.cpp (the pool).  Not installed; the public ABI is
// include/slora.h.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

struct slora_pool;

namespace slora {

constexpr int kKvMaxRequests = 4096;   // == SLORA_KV_MAX_REQUESTS
constexpr int kKvMaxHeadDim = 256;     // == SLORA_KV_MAX_HEAD_DIM
constexpr int kKvRowTile = 8;          // query rows (token, head of the group) of one decode segment
constexpr int kKvUnit = 16;            // tokens of one decode unit
// Warps an SM that a decode kernel of either kind of cache runs at most: each leaves up to two parts of
// split segments in the scratch (kv_attend_parts).
constexpr int kKvDecodeWarps = 12;
// The same of a 4-bit cache: twice as many, with the steps of the softmax once for all of
// them, where registers hold their codes and the result (256 requests of 8 to 640 tokens,
// 32 heads of 128: 115 us with 32 tokens, 129 with 16; 128 of 17 to 8192, 40 heads on 8:
// 165 and 207).
inline int32_t kv_q4_unit(int32_t head_dim) { return head_dim <= 128 ? 2 * kKvUnit : kKvUnit; }
constexpr int kKvTile = 128;           // rows and keys of one chunk tile
// A request whose new tokens make more rows than this (per key head) goes to the
// chunk kernel, which reads the cache once for 256 of them; the decode kernel
// reads it again for every row tile.  16 rows: 128 requests of 17 to 8192
// tokens 368 us against 693, one of 131072 154 against 194, one of 640 14.7
// against 12.3.
constexpr int kKvChunkRows = kKvRowTile;
// Rows of a decode segment of a 4-bit cache, for a call in which no request has more than
// `rows` of them: the kernel works a token's weights out 8 / (rows of a tile) times less
// often with tiles of 2 or 4 (attend_q4.cu).  With chunks in the call the other requests may have
// up to kKvChunkRows, but mostly have one new token, `group` rows.  Tiles by this rule against
// tiles of 8, 128 requests of 17 to 2048 tokens, one row: 32 heads of 64 111 and 123 us, of
// 96 164 and 183, 16 of 160 235 and 248, of 192 229 and 258, of 256 222 and 287; two rows,
// 8 key heads of 224 154 and 182, of 256 119 and 156; four rows, 8 key heads of 64 41 and 45,
// of 96 57 and 61, of 128 59 and 62 (bf16 53 and 58).  256 requests of 8 to 640, 32 heads of
// 128: 115 and 133.  One group alone fills no more columns.
// With chunks the rule is a guess, since a call's lengths are the GPU's to read: the same 128
// requests beside a prompt of 512, 32 heads of 128, with 1 and 2 new tokens each 187 and 191 us
// (214 and 218 with tiles of 8), with 4 and 8, which read the cache two and four times, 332
// and 621 (224 and 230); 4 heads on each of 4, one token 54 and 57, two 73 and 60.
inline int32_t kv_q4_row_tile(int32_t groups, int32_t group, int64_t rows, bool chunks) {
  const int64_t most = chunks ? group : rows;
  if (groups == 1 || most > 4) return kKvRowTile;
  if (groups == 2) return 4;
  return most <= 2 ? 2 : groups <= 4 ? 4 : kKvRowTile;
}
// What a pair of chunk tiles costs besides its key tiles (queries in, results
// out, the first scores waited for), in key tiles' time: about 6,000 cycles
// against 3,000.  Counted with them, the runs of CTAs with many short prompts
// end when the others' do (32 prompts of 8 to 512 tokens: 95 us with 0, 85 with 1, 86 with
// 2 and 3; a 1024-token chunk 261, 259, 259 and 261).
constexpr int kKvPairUnits = 2;
// Query heads per key head the chunk kernel takes: a 128-row tile then holds
// four tokens at least, and a request's tiles stay few enough to be counted
// one by one.
constexpr int kKvChunkGroup = 32;
// Tokens of one row tile of the chunk kernel, 0: this shape runs in the decode
// kernel (head_dim whole 16-element steps of one or two 64-element atoms).
inline int32_t kv_chunk_tokens(int32_t group, int32_t head_dim) {
  return head_dim < 64 || head_dim > 128 || group > kKvChunkGroup ? 0 : kKvTile / group;
}

// Quotients of 31-bit numbers by a fixed divisor (Granlund and Montgomery, "Division
// by Invariant Integers using Multiplication", PLDI 1994): mul = ceil(2^(32 + shift) / d)
// with 2^shift >= d, so that n * mul / 2^(32 + shift) is below 1/d too large
// for every n < 2^32, and the floor is right; mul takes 33 bits, its top bit
// is the extra addition of n.
struct FastDiv {
  uint32_t d = 1, mul = 0, shift = 0;
  void set(uint32_t div) {
    d = div;
    shift = 0;
    while ((1ull << shift) < div) ++shift;
    mul = (uint32_t)((((1ull << shift) - div) << 32) / div + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
#endif
};

// What the kernels of one cache share.  The pool's buffer of a 16-bit cache is
// addressed as a matrix of token rows of heads_kv * head_dim elements: position t
// of a request is row page(t / P) * P + t % P.  In a 4-bit cache the token's row
// begins row_bytes * (t % P) bytes into its page (kv_q4.cuh).
struct KvDev {
  uint16_t* pool;
  int32_t* table;                // [layers][2][max_rows][max_blocks] page of each block, -1: none
  int32_t num_pages;
  int32_t per_page;              // P, tokens per page
  int32_t layers, heads_q, heads_kv, head_dim;
  int32_t max_rows, max_blocks, max_tokens;
  // the planned batch
  int32_t* q_start;              // [R + 1]
  int32_t* kv_len;               // [R] tokens held after the step (0: request left out)
  int32_t* tok_req;              // [T] request of each token, -1: none
  int32_t* tok_pos;              // [T] position of each token in its request
  int4* req;                     // [R] {first token, new tokens, tokens held, table row}, 16-byte aligned
  int32_t* dec_off;              // [R + 1] prefix sums of row tiles * units, the decode kernels' work
  int32_t* tc_off;               // [R + 1] prefix sums of 128-key tiles, the chunk kernel's work per key head
  int32_t* slots;                // [layers][2][max_tokens] pool row of each token, -1: none
  int32_t* error;                // the pool's device error word
  int32_t unit;                  // tokens of one decode unit
  // 4-bit caches
  int32_t groups;                // of 32 elements a head has, 0: a 16-bit cache
  int32_t row_bytes;             // of a token's row
  int64_t page_bytes;
};

struct KvPlanArgs {
  KvDev kv;
  int32_t R, T, max_new;
  int32_t tpt;                   // kv_chunk_tokens
  int32_t row_tile;              // rows of a decode segment
  int32_t tile;                  // tokens a CTA takes at a time (set by the launcher)
  FastDiv per_page_div;
  const int32_t* row;            // NULL: request r has row r
  const int32_t* ctx;
  const int32_t* fresh;          // new tokens per request
  const int32_t* pages;          // [blocks][layers][2]
  int64_t n_blocks;              // blocks `pages` has entries for
};
cudaError_t prepare_kv_kernels();   // opt-in shared memory sizes
cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t st);

struct KvAppendArgs {
  KvDev kv;
  int32_t T, layer;
  const uint16_t *q, *k, *v;
  int64_t ldq, ldk, ldv;
  uint16_t* q_out;
  int64_t ldqo;
  const uint16_t *qw, *kw;       // norm weights [head_dim], NULL: no norm
  float eps;
  const uint64_t* freq;          // [rot_dim / 2] turns a position, in units of 2^-64 turn
  int32_t rot_dim;
  int32_t interleaved;
  float mscale;
  int32_t parts;                 // warps per token (set by the launcher)
  FastDiv per_page_div;          // 4-bit caches
};
cudaError_t launch_kv_append(const KvAppendArgs& a, int dtype, int num_sms, cudaStream_t st);
cudaError_t launch_kv_q4_append(const KvAppendArgs& a, int dtype, int num_sms, cudaStream_t st);

struct KvReadArgs {
  KvDev kv;
  int32_t n, layer;
  const int32_t *row, *pos;      // [n] table row and position of each token, position < 0: none
  uint16_t *k, *v;               // NULL: not wanted
  int64_t ldk, ldv;
  FastDiv per_page_div;
};
cudaError_t launch_kv_read(const KvReadArgs& a, int dtype, cudaStream_t st);

struct KvAttendArgs {
  KvDev kv;
  int32_t R, T, layer;
  const uint16_t* q;
  int64_t ldq;
  uint16_t* out;
  int64_t ldo;
  float scale, softcap;
  float cap_t, cap2;             // softcap > 0: scale / softcap, softcap log2(e)
  float* part_o;                 // parts of split segments: [kv_attend_parts][kv_attend_cols]
  float2* part_ml;               // [kv_attend_parts] their maximum (in powers of two) and sum
  int32_t hbw;                   // neighbouring key heads worked on side by side
  int32_t rows;                  // rows (token, head of the group) a request has at most in the decode kernel
  int32_t row_tile;              // rows of a decode segment
  FastDiv per_page_div;
  // chunk kernel
  int32_t tpt;                   // kv_chunk_tokens
  float* tc_part_o;              // [kv_chunk_part_rows][kKvTile]
  float2* tc_part_ml;
  int4* tc_split;                // per CTA: the split segment that begins in its run
                                 // {first token (-1: none), tokens of tile A << 16 | of tile B, key head, last CTA}
  CUtensorMap q_map;             // q as [T][heads_q][head_dim], box {64, group, tpt}
};
int64_t kv_chunk_part_rows(int num_sms);
cudaError_t prepare_kv_decode_kernels();
cudaError_t prepare_kv_chunk_kernels();
cudaError_t launch_kv_chunk(const KvAttendArgs& a, int dtype, int num_sms, cudaStream_t st);
int64_t kv_attend_parts(int num_sms);
int32_t kv_attend_cols(int32_t head_dim);
// The decode kernel (after_chunks: while the chunk kernel launched before it
// still runs), and the joins of what either kernel split.
cudaError_t launch_kv_decode(const KvAttendArgs& a, int dtype, int num_sms, bool after_chunks, cudaStream_t st);
// (of one type and head size: others are not loaded)
cudaError_t prepare_kv_q4_chunk_kernels(int dtype, int head_dim);
cudaError_t launch_kv_q4_chunk(const KvAttendArgs& a, int dtype, int num_sms, cudaStream_t st);
// The joins alone, of what `groups` groups of CTAs of the 4-bit decode kernel split, with
// the parts' results divided by their sums.
cudaError_t launch_kv_q4_join(const KvAttendArgs& a, int dtype, int num_sms, bool after_chunks, int64_t groups,
                              cudaStream_t st);
// The same over a 4-bit cache.
cudaError_t prepare_kv_q4_decode_kernels(int dtype, int groups);
cudaError_t launch_kv_q4_decode(const KvAttendArgs& a, int dtype, int num_sms, bool after_chunks, cudaStream_t st);

// What kv.cpp uses of a pool (pool.cpp).
struct PoolView {
  uint16_t* d_pool;
  int64_t num_pages;
  int32_t H, dtype, max_tokens, num_sms;
  cudaStream_t compute;
  int32_t* d_error;
  bool planning;
};
PoolView pool_view(const slora_pool* p);
// A tensor map of 16-bit elements, 128-byte swizzle (rank 2 or 3; row strides
// in bytes for the dimensions after the first); the reason is in
// slora_last_error_string().
int encode_map(CUtensorMap* m, const void* base, int dtype, int rank, const uint64_t* dims, const uint64_t* strides,
               const uint32_t* box);
enum KvTimer { kKvTimerPlan = 0, kKvTimerAppend, kKvTimerAttend, kKvTimerRead };
// Brackets a launch with the pool's timing events when timing is on.
struct KvTimed {
  KvTimed(slora_pool* p, KvTimer which);
  void done();
  slora_pool* pool;
  int kind;
  cudaEvent_t start;
};

}  // namespace slora
