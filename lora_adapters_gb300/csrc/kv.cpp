// Host side of the paged key-value cache: argument checks and launches of
// slora_kv_plan, slora_kv_append and slora_kv_attend (include/slora.h).  The
// pages describe the KV half of the unified pool only as an allocation
// (dongaigc.com summary, section 1; fatihsoysal.com page, section "vLLM'in
// PagedAttention Mekanizmasi"); the operators on it are this library's own.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <limits>
#include <new>
#include <vector>

#include "../../include/slora.h"
#include "internal.h"
#include "kv.h"

using namespace slora;

static_assert(kKvMaxRequests == SLORA_KV_MAX_REQUESTS && kKvMaxHeadDim == SLORA_KV_MAX_HEAD_DIM,
              "the public limits are the kernels'");

struct slora_kv {
  slora_pool* pool = nullptr;
  PoolView pv{};
  KvDev dev{};
  uint64_t* d_freq = nullptr;     // rotary turns a position, [head_dim / 2]
  int32_t rot_dim = 0, interleaved = 0;
  float mscale = 1.f;
  float* d_part_o = nullptr;      // the attention's parts of split segments
  float2* d_part_ml = nullptr;
  FastDiv per_page_div;
  int32_t tpt = 0;                // tokens of a chunk tile, 0: the decode kernel takes everything
  float* d_tc_part_o = nullptr;
  float2* d_tc_part_ml = nullptr;
  int4* d_tc_split = nullptr;
  uint64_t generation = 0;
  int32_t R = 0, T = 0, max_new = 0;   // of the planned batch
};

namespace {

// Planned batches of all caches are numbered together: a batch is one cache's alone.
std::atomic<uint64_t> g_generation{0};

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};
#define SLORA_RANGE(name) NvtxRange nvtx_range_(name)

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return code;
}

#define CUDA_TRY(call)                                                            \
  do {                                                                            \
    cudaError_t e_ = (call);                                                      \
    if (e_ != cudaSuccess)                                                        \
      return fail(SLORA_ERR_CUDA, "%s failed: %s", #call, cudaGetErrorString(e_)); \
  } while (0)

void free_kv(slora_kv* kv) {
  cudaFree(kv->d_freq);
  cudaFree(kv->d_part_o);
  cudaFree(kv->d_part_ml);
  cudaFree(kv->d_tc_split);
  cudaFree(kv->d_tc_part_o);
  cudaFree(kv->d_tc_part_ml);
}

// A cache's sizes over a pool: checked, and its KvDev without the arrays.
int check_config(const slora_pool* pool, const slora_kv_config* c, PoolView* pv, KvDev* dev) {
  if (!pool) return fail(SLORA_ERR_INVALID, "pool is NULL");
  if (!c) return fail(SLORA_ERR_INVALID, "config is NULL");
  *pv = pool_view(pool);
  if (pv->planning) return fail(SLORA_ERR_INVALID, "planning pool (no device buffer): no GPU work");
  if (c->layers < 1) return fail(SLORA_ERR_INVALID, "layers=%d", c->layers);
  if (c->heads_kv < 1 || c->heads_q < c->heads_kv || c->heads_q % c->heads_kv)
    return fail(SLORA_ERR_INVALID, "heads_q=%d must be a positive multiple of heads_kv=%d", c->heads_q, c->heads_kv);
  if (c->head_dim < 16 || c->head_dim % 16 || c->head_dim > SLORA_KV_MAX_HEAD_DIM)
    return fail(SLORA_ERR_INVALID, "head_dim=%d must be a multiple of 16 up to %d", c->head_dim,
                SLORA_KV_MAX_HEAD_DIM);
  if (c->max_requests < 1 || c->max_requests > SLORA_KV_MAX_REQUESTS)
    return fail(SLORA_ERR_INVALID, "max_requests=%d not in [1, %d]", c->max_requests, SLORA_KV_MAX_REQUESTS);
  if (c->max_blocks < 1) return fail(SLORA_ERR_INVALID, "max_blocks=%d", c->max_blocks);
  const int64_t width = (int64_t)c->heads_kv * c->head_dim;
  if (pv->H % width)
    return fail(SLORA_ERR_INVALID, "page_elems=%d must be a multiple of heads_kv * head_dim = %lld", pv->H,
                (long long)width);
  const int64_t P = pv->H / width;
  if (pv->num_pages * P >= INT32_MAX || c->max_blocks * P > (1 << 30))
    return fail(SLORA_ERR_INVALID, "more than 2^31 - 2 tokens in the pool, or 2^30 in a table row");
  if ((int64_t)c->heads_q * c->head_dim >= INT32_MAX) return fail(SLORA_ERR_INVALID, "heads_q * head_dim too large");
  KvDev& d = *dev;
  d = KvDev{};
  d.pool = pv->d_pool;
  d.num_pages = (int32_t)pv->num_pages;
  d.per_page = (int32_t)P;
  d.layers = c->layers;
  d.heads_q = c->heads_q;
  d.heads_kv = c->heads_kv;
  d.head_dim = c->head_dim;
  d.max_rows = c->max_requests;
  d.max_blocks = c->max_blocks;
  d.max_tokens = std::max(pv->max_tokens, 1);
  d.error = pv->d_error;
  return SLORA_OK;
}

// Lays the batch arrays out from `base`; the int32 they take.
int64_t place_arrays(KvDev& d, int32_t* base) {
  int32_t* q = base;
  const int64_t T = d.max_tokens, R = d.max_rows;
  d.req = reinterpret_cast<int4*>(q); q += 4 * R;      // first: 16-byte aligned
  d.slots = q; q += (int64_t)2 * d.layers * T;
  d.tok_req = q; q += T;
  d.tok_pos = q; q += T;
  d.q_start = q; q += R + 1;
  d.kv_len = q; q += R;
  d.dec_off = q; q += R + 1;
  d.tc_off = q; q += R + 1;
  return q - base;
}

int check_batch(const slora_kv* kv, const slora_kv_batch* b, int32_t layer) {
  if (!kv) return fail(SLORA_ERR_INVALID, "kv is NULL");
  if (!b || b->generation == 0 || b->generation != kv->generation)
    return fail(SLORA_ERR_INVALID, "the batch is missing, stale (use the last slora_kv_plan's) or another cache's");
  if (layer < 0 || layer >= kv->dev.layers)
    return fail(SLORA_ERR_INVALID, "layer %d not in [0, %d)", layer, kv->dev.layers);
  return SLORA_OK;
}

// A matrix of T rows of `cols` 16-bit elements with row stride ld.
int check_rows(const char* what, const void* p, int64_t ld, int64_t cols) {
  if (!p) return fail(SLORA_ERR_INVALID, "%s is NULL", what);
  if (reinterpret_cast<uintptr_t>(p) & 15) return fail(SLORA_ERR_INVALID, "%s must be 16-byte aligned", what);
  if (ld < cols || ld % 8)
    return fail(SLORA_ERR_INVALID, "%s: row stride %lld must be a multiple of 8 and cover %lld elements", what,
                (long long)ld, (long long)cols);
  return SLORA_OK;
}

// Whether two matrices of T rows of `cols` elements share any.  Rows of one stride are
// compared exactly (slices of one product lie between each other's rows); of two
// strides, only their starts.
bool overlap(const void* p, int64_t ldp, const void* q, int64_t ldq, int64_t cols, int64_t T) {
  if (p == q) return true;
  if (ldp != ldq) return false;
  const int64_t apart = (static_cast<const char*>(q) - static_cast<const char*>(p)) / 2;
  int64_t rows = apart / ldp, off = apart % ldp;
  if (off < 0) {
    off += ldp;
    --rows;
  }
  return (off < cols && std::abs(rows) < T) || (ldp - off < cols && std::abs(rows + 1) < T);
}

}  // namespace

extern "C" {

int slora_kv_array_ints(const slora_pool* pool, const slora_kv_config* c, int64_t* n) {
  SLORA_RANGE("slora_kv_array_ints");
  if (!n) return fail(SLORA_ERR_INVALID, "n is NULL");
  PoolView pv;
  KvDev d;
  if (int rc = check_config(pool, c, &pv, &d)) return rc;
  *n = place_arrays(d, nullptr);
  return SLORA_OK;
}

int slora_kv_create(slora_kv** out, slora_pool* pool, const slora_kv_config* c, int32_t* d_table,
                    int32_t* d_arrays) {
  SLORA_RANGE("slora_kv_create");
  if (!out) return fail(SLORA_ERR_INVALID, "out is NULL");
  *out = nullptr;
  PoolView pv;
  KvDev d;
  if (int rc = check_config(pool, c, &pv, &d)) return rc;
  if (!d_table || !d_arrays || reinterpret_cast<uintptr_t>(d_table) & 3 || reinterpret_cast<uintptr_t>(d_arrays) & 15)
    return fail(SLORA_ERR_INVALID, "d_table and d_arrays must be device pointers to int32, d_arrays 16-byte aligned");

  slora_kv* kv = new (std::nothrow) slora_kv();
  if (!kv) return fail(SLORA_ERR_OOM, "host allocation failed");
  d.table = d_table;
  const int64_t ints = place_arrays(d, d_arrays);
  kv->pool = pool;
  kv->pv = pv;
  kv->dev = d;
  kv->per_page_div.set((uint32_t)d.per_page);
  auto setup = [&]() -> int {
    CUDA_TRY(prepare_kv_kernels());
    CUDA_TRY(prepare_kv_decode_kernels());
    CUDA_TRY(cudaMalloc(&kv->d_freq, sizeof(uint64_t) * (size_t)(c->head_dim / 2)));
    const int64_t parts = kv_attend_parts(pv.num_sms);
    CUDA_TRY(cudaMalloc(&kv->d_part_o, sizeof(float) * (size_t)parts * (size_t)kv_attend_cols(c->head_dim)));
    CUDA_TRY(cudaMalloc(&kv->d_part_ml, sizeof(float2) * (size_t)parts));
    kv->tpt = kv_chunk_tokens(d.heads_q / d.heads_kv, d.head_dim);
    if (kv->tpt > 0) {
      CUDA_TRY(prepare_kv_chunk_kernels());
      const int64_t rows = kv_chunk_part_rows(pv.num_sms);
      CUDA_TRY(cudaMalloc(&kv->d_tc_part_o, sizeof(float) * (size_t)rows * kKvTile));
      CUDA_TRY(cudaMalloc(&kv->d_tc_part_ml, sizeof(float2) * (size_t)rows));
      CUDA_TRY(cudaMalloc(&kv->d_tc_split, sizeof(int4) * (size_t)pv.num_sms));
    }
    CUDA_TRY(cudaMemsetAsync(d_arrays, 0, sizeof(int32_t) * (size_t)ints, pv.compute));
    CUDA_TRY(cudaMemsetAsync(d_table, 0xff,
                             sizeof(int32_t) * (size_t)2 * c->layers * (size_t)c->max_requests * (size_t)c->max_blocks,
                             pv.compute));
    return SLORA_OK;
  };
  const int rc = setup();
  if (rc != SLORA_OK) {
    (void)cudaStreamSynchronize(pv.compute);
    free_kv(kv);
    delete kv;
    return rc;
  }
  *out = kv;
  return SLORA_OK;
}

int slora_kv_destroy(slora_kv* kv) {
  SLORA_RANGE("slora_kv_destroy");
  if (!kv) return fail(SLORA_ERR_INVALID, "kv is NULL");
  int rc = SLORA_OK;
  const cudaError_t e = cudaStreamSynchronize(kv->pv.compute);
  if (e != cudaSuccess) rc = fail(SLORA_ERR_CUDA, "stream synchronize at destroy: %s", cudaGetErrorString(e));
  free_kv(kv);
  delete kv;
  return rc;
}

int slora_kv_set_rotary(slora_kv* kv, int32_t rot_dim, int32_t layout, const double* h_inv_freq, float mscale) {
  SLORA_RANGE("slora_kv_set_rotary");
  if (!kv) return fail(SLORA_ERR_INVALID, "kv is NULL");
  if (rot_dim < 0 || rot_dim % 16 || rot_dim > kv->dev.head_dim)
    return fail(SLORA_ERR_INVALID, "rot_dim=%d must be a multiple of 16 up to head_dim=%d", rot_dim, kv->dev.head_dim);
  if (layout != SLORA_ROTARY_HALF && layout != SLORA_ROTARY_INTERLEAVED)
    return fail(SLORA_ERR_INVALID, "layout %d", layout);
  if (rot_dim > 0 && !h_inv_freq) return fail(SLORA_ERR_INVALID, "h_inv_freq is NULL");
  if (!std::isfinite(mscale)) return fail(SLORA_ERR_INVALID, "mscale is not finite");
  uint64_t turns[kKvMaxHeadDim / 2];
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (!std::isfinite(h_inv_freq[i])) return fail(SLORA_ERR_INVALID, "frequency %d is not finite", i);
    // turns a position, its whole part dropped, as a fraction of 2^64.  The
    // quotient's 53 bits are split so that the conversion keeps all of them
    double f = h_inv_freq[i] / 6.283185307179586476925286766559;
    f -= std::floor(f);
    const double hi = std::floor(std::ldexp(f, 32));
    const double lo = std::ldexp(f, 64) - std::ldexp(hi, 32);
    turns[i] = ((uint64_t)std::min(hi, 4294967296.0) << 32) + (uint64_t)lo;
  }
  if (rot_dim > 0) {
    // `turns` is pageable: the copy is staged before the call returns, and it
    // is ordered after the appends queued so far
    CUDA_TRY(cudaMemcpyAsync(kv->d_freq, turns, sizeof(uint64_t) * (size_t)(rot_dim / 2), cudaMemcpyHostToDevice,
                             kv->pv.compute));
    CUDA_TRY(cudaStreamSynchronize(kv->pv.compute));
  }
  kv->rot_dim = rot_dim;
  kv->interleaved = layout == SLORA_ROTARY_INTERLEAVED;
  kv->mscale = mscale;
  return SLORA_OK;
}

int slora_kv_plan(slora_kv* kv, int32_t R, const int32_t* d_row, const int32_t* d_ctx, const int32_t* d_new,
                  const int32_t* d_pages, int64_t n_pages, int32_t T, int32_t max_new, slora_kv_batch* out) {
  SLORA_RANGE("slora_kv_plan");
  if (!kv) return fail(SLORA_ERR_INVALID, "kv is NULL");
  if (!out) return fail(SLORA_ERR_INVALID, "out is NULL");
  if (R < 0 || R > kv->dev.max_rows) return fail(SLORA_ERR_INVALID, "R=%d not in [0, %d]", R, kv->dev.max_rows);
  if (T < 0 || T > kv->pv.max_tokens) return fail(SLORA_ERR_INVALID, "T=%d not in [0, %d]", T, kv->pv.max_tokens);
  if (max_new < 0) return fail(SLORA_ERR_INVALID, "max_new=%d", max_new);
  if (R > 0 && (!d_ctx || !d_new)) return fail(SLORA_ERR_INVALID, "NULL lengths");
  if (n_pages < 0 || n_pages % (2 * kv->dev.layers) || (n_pages > 0 && !d_pages))
    return fail(SLORA_ERR_INVALID, "n_pages=%lld must be whole blocks of 2 * layers pages, d_pages not NULL",
                (long long)n_pages);
  if ((reinterpret_cast<uintptr_t>(d_row) | reinterpret_cast<uintptr_t>(d_ctx) | reinterpret_cast<uintptr_t>(d_new) |
       reinterpret_cast<uintptr_t>(d_pages)) & 3)
    return fail(SLORA_ERR_INVALID, "device arrays must be aligned int32");
  KvPlanArgs a{};
  a.kv = kv->dev;
  a.R = R;
  a.T = T;
  a.max_new = max_new;
  a.tpt = kv->tpt;
  a.per_page_div = kv->per_page_div;
  a.row = d_row;
  a.ctx = d_ctx;
  a.fresh = d_new;
  a.pages = d_pages;
  a.n_blocks = n_pages / (2 * kv->dev.layers);
  {
    KvTimed tm(kv->pool, kKvTimerPlan);
    CUDA_TRY(launch_kv_plan(a, kv->pv.compute));
    tm.done();
  }
  kv->generation = ++g_generation;
  kv->R = R;
  kv->T = T;
  kv->max_new = max_new;
  const KvDev& d = kv->dev;
  *out = slora_kv_batch{R, T, max_new, d.q_start, d.kv_len, d.tok_req, d.tok_pos, d.slots, d.max_tokens,
                        kv->generation};
  return SLORA_OK;
}

int slora_kv_append(slora_kv* kv, const slora_kv_batch* batch, int32_t layer, const void* d_q, int64_t ldq,
                    const void* d_k, int64_t ldk, const void* d_v, int64_t ldv, const void* d_q_weight,
                    const void* d_k_weight, float eps, void* d_q_out, int64_t ldqo) {
  SLORA_RANGE("slora_kv_append");
  if (int rc = check_batch(kv, batch, layer)) return rc;
  if (kv->T == 0) return SLORA_OK;
  const KvDev& d = kv->dev;
  const int64_t wq = (int64_t)d.heads_q * d.head_dim, wk = (int64_t)d.heads_kv * d.head_dim;
  if (int rc = check_rows("q", d_q, ldq, wq)) return rc;
  if (int rc = check_rows("k", d_k, ldk, wk)) return rc;
  if (int rc = check_rows("v", d_v, ldv, wk)) return rc;
  if (int rc = check_rows("q_out", d_q_out, ldqo, wq)) return rc;
  if (d_q_out == d_q && ldqo != ldq) return fail(SLORA_ERR_INVALID, "q_out in place needs q's row stride");
  if (d_q_out != d_q && overlap(d_q, ldq, d_q_out, ldqo, wq, kv->T))
    return fail(SLORA_ERR_INVALID, "q_out overlaps q");
  if (!d_q_weight != !d_k_weight) return fail(SLORA_ERR_INVALID, "norm weights of queries and keys go together");
  if ((reinterpret_cast<uintptr_t>(d_q_weight) | reinterpret_cast<uintptr_t>(d_k_weight)) & 15)
    return fail(SLORA_ERR_INVALID, "norm weights must be 16-byte aligned");
  if (d_q_weight && !(std::isfinite(eps) && eps >= 0.f)) return fail(SLORA_ERR_INVALID, "eps must be finite and >= 0");
  KvAppendArgs a{};
  a.kv = d;
  a.T = kv->T;
  a.layer = layer;
  a.q = static_cast<const uint16_t*>(d_q);
  a.k = static_cast<const uint16_t*>(d_k);
  a.v = static_cast<const uint16_t*>(d_v);
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.q_out = static_cast<uint16_t*>(d_q_out);
  a.ldqo = ldqo;
  a.qw = static_cast<const uint16_t*>(d_q_weight);
  a.kw = static_cast<const uint16_t*>(d_k_weight);
  a.eps = eps;
  a.freq = kv->d_freq;
  a.rot_dim = kv->rot_dim;
  a.interleaved = kv->interleaved;
  a.mscale = kv->mscale;
  KvTimed tm(kv->pool, kKvTimerAppend);
  CUDA_TRY(launch_kv_append(a, kv->pv.dtype, kv->pv.num_sms, kv->pv.compute));
  tm.done();
  return SLORA_OK;
}

int slora_kv_attend(slora_kv* kv, const slora_kv_batch* batch, int32_t layer, const void* d_q, int64_t ldq,
                    void* d_out, int64_t ldo, float scale, float softcap) {
  SLORA_RANGE("slora_kv_attend");
  if (int rc = check_batch(kv, batch, layer)) return rc;
  if (!std::isfinite(scale) || scale <= 0.f) return fail(SLORA_ERR_INVALID, "scale must be finite and > 0");
  if (!std::isfinite(softcap) || softcap < 0.f) return fail(SLORA_ERR_INVALID, "softcap must be finite and >= 0");
  if (kv->T == 0 || kv->R == 0 || kv->max_new == 0) return SLORA_OK;   // no request can have a row
  const int32_t group = kv->dev.heads_q / kv->dev.heads_kv;
  const int64_t rows = (int64_t)std::min(kv->max_new, kv->T) * group;     // of one key head in one request
  // chunks are possible where one request may bring more than kKvChunkRows rows
  const bool chunks = kv->tpt > 0 && rows > kKvChunkRows;
  if (!chunks && rows * kv->dev.heads_kv > INT32_MAX)
    return fail(SLORA_ERR_INVALID, "max_new * heads_q = %lld is 2^31 or more", (long long)rows * kv->dev.heads_kv);
  const int64_t wq = (int64_t)kv->dev.heads_q * kv->dev.head_dim;
  if (int rc = check_rows("q", d_q, ldq, wq)) return rc;
  if (int rc = check_rows("out", d_out, ldo, wq)) return rc;
  if (overlap(d_q, ldq, d_out, ldo, wq, kv->T)) return fail(SLORA_ERR_INVALID, "out overlaps q");
  KvAttendArgs a{};
  a.kv = kv->dev;
  a.R = kv->R;
  a.T = kv->T;
  a.layer = layer;
  a.q = static_cast<const uint16_t*>(d_q);
  a.ldq = ldq;
  a.out = static_cast<uint16_t*>(d_out);
  a.ldo = ldo;
  a.scale = scale;
  a.softcap = softcap;
  if (softcap > 0.f) {   // kept finite, four times each too: a product q . k of 0 has the score 0 at every softcap
    const double most = std::numeric_limits<float>::max() / 4;
    a.cap_t = (float)std::min((double)scale / softcap, most);
    a.cap2 = (float)std::min((double)softcap * 1.4426950408889634, most);
  }
  a.part_o = kv->d_part_o;
  a.part_ml = kv->d_part_ml;
  a.tc_split = kv->d_tc_split;
  a.per_page_div = kv->per_page_div;
  a.tpt = kv->tpt;
  a.tc_part_o = kv->d_tc_part_o;
  a.tc_part_ml = kv->d_tc_part_ml;
  a.rows = chunks ? kKvChunkRows : (int32_t)rows;
  if (chunks) {
    const uint64_t dims[3] = {(uint64_t)kv->dev.head_dim, (uint64_t)kv->dev.heads_q, (uint64_t)kv->T};
    const uint64_t strides[2] = {2 * (uint64_t)kv->dev.head_dim, 2 * (uint64_t)ldq};
    const uint32_t box[3] = {64, (uint32_t)group, (uint32_t)kv->tpt};
    if (int rc = encode_map(&a.q_map, d_q, kv->pv.dtype, 3, dims, strides, box)) return rc;
  }
  KvTimed tm(kv->pool, kKvTimerAttend);
  if (chunks) CUDA_TRY(launch_kv_chunk(a, kv->pv.dtype, kv->pv.num_sms, kv->pv.compute));
  CUDA_TRY(launch_kv_decode(a, kv->pv.dtype, kv->pv.num_sms, chunks, kv->pv.compute));
  tm.done();
  return SLORA_OK;
}

}  // extern "C"
