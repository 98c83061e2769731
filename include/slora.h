/*
 * slora.h -- C ABI of the GB300 heterogeneous-batch LoRA library (libslora.so).
 *
 * The library implements the data-parallel hot path of S-LoRA ("S-LoRA:
 * Serving Thousands of Concurrent LoRA Adapters", MLSys 2024): for every
 * token i of one batch, with its own adapter a = a(i) of its own rank r_a,
 *
 *     y_i  +=  s * (x_i A_a) B_a
 *
 * where the rows of A_a and B_a are not contiguous tensors but sit on pages
 * of one unified pool that the adapters share with the KV cache.
 *   - Unified Paging: one pool of fixed-size pages holds adapter weights of
 *     different ranks and KV tensors of different lengths (nubint.ai review,
 *     abstract and method list; dongaigc.com summary, section 1).
 *   - Adapters live in host memory and are fetched to the GPU on demand,
 *     asynchronously (nubint.ai review, abstract; cmlonder.com newsletter,
 *     section "Iddia ve Gerceklik").
 *   - Heterogeneous batching: one pass computes the LoRA part for tokens of
 *     many adapters of different ranks directly on non-contiguous memory
 *     (dongaigc.com summary, section 2; nubint.ai review, method list).
 *   - The base model's batched GEMM is computed elsewhere; this library only
 *     adds the adapter part into its output y (nubint.ai review, method list:
 *     base computation batched, adapter computation separate).
 *
 * Conventions for every function below
 *   - Return value: SLORA_OK (0) or a negative SLORA_ERR_* code.  On error
 *     nothing observable changed (allocator state, page tables, device data)
 *     unless the description says otherwise; slora_last_error_string() then
 *     holds a one-line reason (thread-local, valid until the next call on
 *     the same thread).
 *   - "device pointer" = memory of the GPU current when the pool was
 *     created; "host pointer" = ordinary (preferably pinned) host memory.
 *   - Streams/events are cudaStream_t / cudaEvent_t passed as void*.  All
 *     device work of the pool is ordered on its compute stream, except
 *     adapter copies, which run on its copy stream.  No function blocks the
 *     host on the GPU unless it says so.
 *   - A pool is not thread-safe: the caller serialises calls on one pool.
 *   - 16-bit values are IEEE binary16 (SLORA_F16) or bfloat16 (SLORA_BF16);
 *     accumulation is fp32; y is rounded once, to nearest even.
 */
#ifndef SLORA_H
#define SLORA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define SLORA_OK 0
#define SLORA_ERR_INVALID (-1)      /* bad argument, size, alignment or id */
#define SLORA_ERR_OOM (-2)          /* not enough free pages; state unchanged */
#define SLORA_ERR_EXISTS (-3)       /* adapter id already resident */
#define SLORA_ERR_NOT_RESIDENT (-4) /* adapter id not resident */
#define SLORA_ERR_BUSY (-5)         /* reserved, never returned: an evict of an adapter still in use
                                       is ordered by events instead (see slora_adapter_evict) */
#define SLORA_ERR_CUDA (-6)         /* a CUDA runtime call failed (see error string) */
#define SLORA_ERR_DEVICE (-7)       /* a kernel reported bad input (see slora_device_status) */
#define SLORA_ERR_TIMEOUT (-8)      /* a kernel's bounded wait gave up (device status only) */
#define SLORA_ERR_DEVICE_ASSERT (-9) /* a bounds check of the SLORA_DEBUG build failed (device status only) */

/* ---- element types and apply modes -------------------------------------- */
#define SLORA_F16 0
#define SLORA_BF16 1

#define SLORA_MODE_AUTO 0    /* large batches: tcgen05 for long segments, CUDA cores for the rest; small batches: CUDA cores */
#define SLORA_MODE_DECODE 1  /* every segment on the CUDA-core gather kernels */
#define SLORA_MODE_PREFILL 2 /* every segment on the tcgen05 kernels (CUDA-core kernels when the page size is not a multiple of 64) */

/* Library limits (also checked at run time). */
#define SLORA_MAX_PROJ 128         /* projections per pool (e.g. 32 layers x q, k, v, o) */
#define SLORA_MAX_PROJ_PER_CALL 8  /* projections of one slora_lora_apply_multi call */
#define SLORA_MAX_RANK 256         /* largest adapter rank */
#define SLORA_MAX_ADAPTERS 32768   /* adapter ids 0 .. max_adapters-1 */

typedef struct slora_pool slora_pool; /* opaque, owned by the library */

/*
 * The token grouping of one batch (the "segments" of segmented gather
 * matrix-vector products, SGMV: cmlonder.com newsletter, section "Iddia ve
 * Gerceklik").  Tokens are stably sorted by adapter id, ascending; tokens
 * with id -1 carry no adapter and are left out, as are tokens that name an
 * adapter that is not resident or an id outside [-1, max_adapters) (those
 * are counted in counts[2] and raise the device status
 * SLORA_ERR_NOT_RESIDENT or SLORA_ERR_INVALID; the first such token seen
 * decides which).  All arrays are DEVICE memory
 * owned by the pool; they stay valid until the next slora_build_segments on
 * the same pool (or the next evict), which invalidates every earlier handle
 * (generation check).
 */
typedef struct slora_segments {
  int32_t T;                  /* tokens in the batch */
  int32_t max_segs;           /* capacity of seg_adapter / seg_start */
  const int32_t* perm;        /* [T] sorted position j -> token index; [0, counts[1]) valid */
  const int32_t* seg_start;   /* [max_segs + 1] first sorted position of each segment */
  const int32_t* seg_adapter; /* [max_segs] adapter id of each segment (ascending) */
  const int32_t* counts;      /* [16] {num_segs, n_sorted, bad_tokens, internal work totals...} */
  uint64_t generation;        /* must match the pool's current segment generation */
} slora_segments;

/*
 * Create a pool over a caller-owned device buffer.  The pool is the unified
 * memory pool of S-LoRA's Unified Paging (dongaigc.com summary, section 1
 * "Unified Paging": one pool of pages managed together for adapter weights
 * and KV-cache tensors; nubint.ai review, method list): pages of H elements,
 * the unit one token's K or V vector of one layer takes, so that adapter rows
 * of every rank and KV slots of every length are allocated from one free list
 * without fragmenting it.
 *   d_pool      device buffer of num_pages * page_elems 16-bit elements,
 *               16-byte aligned; caller-owned, must outlive the pool.  NULL
 *               creates a PLANNING pool: host allocator and page tables only,
 *               no CUDA call is ever made (loads only allocate; build/apply
 *               return SLORA_ERR_INVALID).
 *   num_pages   pages in the pool (> 0, < 2^31)
 *   page_elems  H = elements per page = the hidden size = one token's K (or
 *               V) vector for one layer, so one KV slot of one token and one
 *               layer is two pages; multiple of 8, <= 65536
 *   dtype       SLORA_F16 or SLORA_BF16 (pool, x and y share it)
 *   max_adapters, max_rank   adapter ids are 0..max_adapters-1, ranks 1..max_rank
 *   max_tokens  largest batch (T) accepted by slora_build_segments
 *   num_proj, proj_in, proj_out   the projections adapters carry (host
 *               arrays, copied); every dim a positive multiple of 8
 *   compute, copy   cudaStream_t for kernels / for adapter copies (may be
 *               equal; NULL = legacy default stream)
 * Allocates with cudaMalloc: the device page table (max_adapters * max_rank
 * * sum_q(ceil(in_q/H)+ceil(out_q/H)) int32), segment arrays, the fp32
 * shrink scratch (SLORA_MAX_PROJ_PER_CALL * max_tokens * max_rank floats) and one
 * adapter-sized staging buffer; pins an equally sized host page-table mirror.
 */
int slora_pool_create(slora_pool** out, void* d_pool, int64_t num_pages, int32_t page_elems,
                      int32_t dtype, int32_t max_adapters, int32_t max_rank, int32_t max_tokens,
                      int32_t num_proj, const int32_t* proj_in, const int32_t* proj_out,
                      void* compute_stream, void* copy_stream);

/* Synchronises both streams and frees everything the pool allocated (not d_pool). */
int slora_pool_destroy(slora_pool* pool);

/*
 * KV-slot pages (PagedAttention-style: taken on demand, returned when a
 * request ends; fatihsoysal.com page, section "vLLM'in PagedAttention
 * Mekanizmasi").  alloc writes the n lowest-numbered free pages, ascending,
 * to out_pages (host int32[n]); all or nothing (SLORA_ERR_OOM).  free
 * returns n KV pages (host int32[n]); every page must be a KV page and
 * listed once, else SLORA_ERR_INVALID and nothing is freed.  Pages released
 * by slora_adapter_evict may still be read by kernels already queued on the
 * compute stream: write reused pages on that stream or after it.
 */
int slora_pages_alloc(slora_pool* pool, int64_t n, int32_t* out_pages);
int slora_pages_free(slora_pool* pool, int64_t n, const int32_t* pages);

/* Free page count and page size; any pointer may be NULL. */
int slora_pool_info(const slora_pool* pool, int64_t* free_pages, int64_t* num_pages,
                    int32_t* page_elems, int64_t* pages_per_rank);

/*
 * Load adapter `adapter_id` of rank `rank` from host memory into pool pages
 * (the on-demand fetch of the nubint.ai review, abstract).  Allocates
 * rank * sum_q(ceil(in_q/H) + ceil(out_q/H)) pages, lowest-numbered first,
 * and lists them in this page-table order: for each projection q, the rank
 * rows of A (each ceil(in_q/H) page chunks), then the rank rows of B (each
 * ceil(out_q/H) chunks); the i-th lowest page holds the i-th chunk.  The tail
 * of a row's last page is zero-filled.
 *   h_A[q]  host, rank x in_q 16-bit row-major: row k is column k of the
 *           in_q x rank matrix A (A transposed)
 *   h_B[q]  host, rank x out_q 16-bit row-major: row k is row k of B
 *   done    optional out: a cudaEvent_t (owned by the pool, valid until the
 *           adapter is evicted) that completes when the pages are written
 * The copies are queued on the copy stream after all work queued so far on
 * the compute stream (so pages freed earlier are no longer being read; weight
 * blocks that follow each other in host memory in the order above move in one
 * copy) and
 * the host buffers must stay untouched until `done` completes.  Later
 * slora_build_segments calls make the compute stream wait for pending loads.
 * Errors: SLORA_ERR_INVALID (id/rank out of range, NULL buffer),
 * SLORA_ERR_EXISTS, SLORA_ERR_OOM (state unchanged), SLORA_ERR_CUDA (the
 * pages are released again, state as before the call).
 * On a planning pool h_A / h_B may be NULL and nothing is copied.
 */
int slora_adapter_load(slora_pool* pool, int32_t adapter_id, int32_t rank,
                       const void* const* h_A, const void* const* h_B, void** done);

/*
 * Evict a resident adapter: its pages return to the free list at once and
 * its device rank is cleared on the compute stream (work queued before the
 * evict still sees the adapter; if the adapter's load is still copying, work
 * queued on the compute stream after the evict waits for those copies).  The pages' "race conditions in the adapter
 * manager under dynamic loading" (cmlonder.com newsletter, section "Iddia ve
 * Gerceklik") are answered by stream order rather than by refusing the evict
 * with SLORA_ERR_BUSY: a later load into the freed pages is queued after all
 * work queued on the compute stream before it, so no kernel still reading the
 * old rows can see the new ones.  Every segment handle built before the
 * evict becomes stale (build the segments again).  SLORA_ERR_NOT_RESIDENT if
 * it is not loaded.
 */
int slora_adapter_evict(slora_pool* pool, int32_t adapter_id);

/*
 * Per-adapter scale s_a (LoRA's alpha / r): applies compute
 *     y += s * s_a * (x A_a) B_a
 * for tokens of adapter a.  A load sets s_a = 1; this call changes it for
 * applies queued on the compute stream after it (it waits for the adapter's
 * own pending load first).  Errors: SLORA_ERR_NOT_RESIDENT for an adapter
 * that is not loaded, SLORA_ERR_INVALID for a scale that is not finite, and
 * for a planning pool (no device state).
 */
int slora_adapter_set_scale(slora_pool* pool, int32_t adapter_id, float scale);

/*
 * *ready = 1 once adapter `adapter_id`'s load has finished on the copy
 * stream (always on a planning pool), 0 while its copies are still running;
 * never blocks.  A scheduler that admits a request only when its adapter is
 * ready keeps slora_build_segments from making the compute stream wait for
 * copies (it waits for every load still running).  SLORA_ERR_NOT_RESIDENT if
 * the adapter is not loaded.
 */
int slora_adapter_ready(slora_pool* pool, int32_t adapter_id, int32_t* ready);

/* Host copy of an adapter's page table (page-table order above); *n = entries. */
int slora_adapter_pages(const slora_pool* pool, int32_t adapter_id, int32_t* out_pages,
                        int64_t capacity, int64_t* n);

/*
 * Group the batch's tokens by adapter on the GPU (one kernel on the compute
 * stream).  d_token_adapter: device int32[T], ids in [-1, max_adapters);
 * 0 <= T <= max_tokens.  Fills *out with pool-owned device arrays (see
 * slora_segments) plus the internal work lists of the apply kernels.
 *
 * CUDA graphs: this call and the apply calls only enqueue work on the
 * compute stream, so a step (segments, then one apply per layer) can be
 * captured in a graph and replayed, as long as the compute stream is not
 * the legacy default stream and no load of an adapter the batch uses is
 * still copying when the capture is made (its wait would refer to a copy
 * outside the graph).  A replay rebuilds the segments from the token ids
 * then in the captured buffer.
 */
int slora_build_segments(slora_pool* pool, const int32_t* d_token_adapter, int32_t T,
                         slora_segments* out);

/*
 * The same, for a caller that also holds the batch's ids on the host (a
 * scheduler builds them there): h_token_adapter, host int32[T], must list the
 * same ids as d_token_adapter.  The compute stream then waits only for the
 * pending loads of the adapters the batch names, not for every pending load
 * -- a load started for a request that has not joined the batch yet does not
 * hold this batch back.  h_token_adapter NULL: as slora_build_segments.
 */
int slora_build_segments_for(slora_pool* pool, const int32_t* d_token_adapter, int32_t T,
                             const int32_t* h_token_adapter, slora_segments* out);

/*
 * The heterogeneous-batch LoRA delta (dongaigc.com summary, section 2
 * "Heterogeneous Batching": the adapter part of tokens that use different
 * adapters of different ranks computed in one pass by custom kernels that
 * read the weights directly from the non-contiguous pool; cmlonder.com
 * newsletter, section "Iddia ve Gerceklik": segmented gather kernels, SGMV):
 * y += s * (x A_a) B_a for one projection `proj` over every token of the
 * batch `seg` was built from (tokens left out of the segments are not
 * touched).  x: device, T rows of proj_in[proj] elements, row stride ldx
 * elements; y: device, T rows of proj_out[proj], stride ldy, updated in
 * place.  Strides multiples of 8, pointers 16-byte aligned, x and y must not
 * overlap.  mode: SLORA_MODE_*.  Kernels only; nothing is synchronised.
 */
int slora_lora_apply(slora_pool* pool, const slora_segments* seg, int32_t proj, const void* d_x,
                     int64_t ldx, void* d_y, int64_t ldy, float s, int32_t mode);

/* The same for n <= SLORA_MAX_PROJ_PER_CALL projections (e.g. one layer's
 * q, k, v, o) in one set of launches. */
int slora_lora_apply_multi(slora_pool* pool, const slora_segments* seg, int32_t n,
                           const int32_t* projs, const void* const* d_x, const int64_t* ldx,
                           void* const* d_y, const int64_t* ldy, float s, int32_t mode);

/*
 * Comparator: the same delta by the "traditional batched matmul" variant
 * that the pages compare S-LoRA with (dongaigc.com summary, section
 * "S-LoRA的性能评估": S-LoRA against its own variants, one without unified
 * memory, one with traditional batched matrix multiplication).  Every token's
 * adapter rows are gathered out of the pool into dense tensors padded to the
 * pool's max_rank (zeros past the adapter's rank), two cuBLAS strided-batched
 * GEMMs give (x_t A) B per token (fp32 accumulation, v kept in fp32), and
 * y_t += s * s_a * delta_t is rounded once.  Arguments and errors as
 * slora_lora_apply (one projection; no mode).  Scratch: on the first call
 * the pool allocates max_tokens * max_rank * (2 * max h_in + 4 * max h_out)
 * bytes and a little more (slora_bmm_scratch_bytes reports it), freed with
 * the pool; SLORA_ERR_OOM if it cannot.  cuBLAS is opened on the first call
 * (SLORA_ERR_CUDA when it is not installed); nothing else in the library
 * needs it.  For measurement and comparison, not for serving.
 */
int slora_lora_apply_bmm(slora_pool* pool, const slora_segments* seg, int32_t proj, const void* d_x,
                         int64_t ldx, void* d_y, int64_t ldy, float s);
/* Bytes of comparator scratch the pool holds (0 before the first call). */
int slora_bmm_scratch_bytes(const slora_pool* pool, size_t* bytes);

/*
 * Synchronises the compute stream, returns in *status the first error a
 * kernel reported since the last call (SLORA_OK, SLORA_ERR_NOT_RESIDENT for a
 * token naming an adapter that is not loaded, SLORA_ERR_INVALID for an id
 * out of range, SLORA_ERR_TIMEOUT when a pipeline wait gave up) and clears it.
 */
int slora_device_status(slora_pool* pool, int32_t* status);

/*
 * Serialise the host allocator state for bit-exact comparison: int64
 * num_pages, int64 free_pages, int32 max_adapters, int32 stride, then
 * int32 owner[num_pages] (-1 free, -2 KV, else adapter id), int32
 * rank[max_adapters], int32 page_table[max_adapters * stride] (-1 unused).
 * With buf NULL only *len is set; otherwise *len must be >= the size.
 */
int slora_pool_snapshot(const slora_pool* pool, void* buf, size_t* len);

/*
 * Per-kernel device timing (tracing).  When enabled, every kernel the pool
 * launches is bracketed by CUDA events on its stream.  slora_timing_read
 * synchronises, then writes for each kernel kind k < *n (at most capacity):
 * names[k] (static strings), total milliseconds ms[k] and launches[k], and
 * resets the totals.
 */
int slora_timing_enable(slora_pool* pool, int32_t enable);
int slora_timing_read(slora_pool* pool, int32_t capacity, const char** names, double* ms,
                      int64_t* launches, int32_t* n);

/*
 * SLORA_MODE_AUTO's split.  In a batch of at least `tc_min_batch` tokens
 * (default 2048), segments of at least `tc_threshold` tokens (default 8) run
 * on the tcgen05 kernels and the rest on the CUDA-core kernel; a smaller
 * batch runs wholly on the CUDA-core kernel.  The defaults come from
 * measurements on GB300: on the 7B prefill batch (8,561 tokens) AUTO then
 * matches PREFILL, while on decode batches of 256-512 tokens the few long
 * segments leave the tensor-core kernels bound by latency and the CUDA-core
 * kernel is 1.8x faster.  tc_threshold takes effect at the next
 * slora_build_segments; tc_min_batch at the next apply.
 */
int slora_set_tc_threshold(slora_pool* pool, int32_t min_tokens);
int slora_set_tc_min_batch(slora_pool* pool, int32_t min_tokens);

/*
 * Failure injection on the host, for tests of the error paths (the pages'
 * concern about the adapter manager under dynamic loading: cmlonder.com
 * newsletter, section "Iddia ve Gerceklik").  Arms one fault on this pool;
 * it fires once, on the nth (counted from 1) event of its kind from now on:
 *   SLORA_FAULT_PAGE_ALLOC  a call that takes pages (slora_pages_alloc,
 *                           slora_adapter_load) fails with SLORA_ERR_OOM as
 *                           if the pool were full; nothing changes;
 *   SLORA_FAULT_COPY        a copy or kernel that slora_adapter_load enqueues
 *                           fails as a CUDA error would: the load returns
 *                           SLORA_ERR_CUDA and, once the copy stream has
 *                           finished what the load queued before the failure,
 *                           its pages are released again, the host state
 *                           (slora_pool_snapshot) exactly as before the call.
 * SLORA_FAULT_NONE (or nth = 0) disarms.  The environment variable
 * SLORA_FAULT="alloc:N" or "copy:N" arms the same fault in every pool the
 * process creates.  Nothing here touches a GPU.
 */
#define SLORA_FAULT_NONE 0
#define SLORA_FAULT_PAGE_ALLOC 1
#define SLORA_FAULT_COPY 2
int slora_debug_set_fault(slora_pool* pool, int32_t kind, int64_t nth);

/*
 * The SLORA_DEBUG build (libslora_debug.so, compiled with -DSLORA_DEBUG;
 * the Python binding loads it when the environment has SLORA_DEBUG=1)
 * checks, in every kernel, each page index it reads from a page table
 * against the pool's page count and each token index it reads from the
 * token order against the batch size.  A violation is reported by
 * slora_device_status as SLORA_ERR_DEVICE_ASSERT (the index is replaced by
 * 0, so no access leaves its buffer and no kernel waits for a copy that
 * never comes); results of that call are then meaningless.  Other builds
 * compile no checks.  slora_kv_append checks the slots, slora_kv_attend the
 * table rows and token indices that they read from a planned batch's arrays;
 * pages of the block table are checked in every build (slora_kv_plan and
 * slora_kv_attend).
 *
 * slora_debug_poke_page_table writes `value` into entry `entry` of the
 * pool's device page table (entries of adapter a start at a * stride) and
 * returns the previous value in *old: a test plants a bad page index and
 * puts the old one back.  The host copy of the table is not changed.  Only
 * in the SLORA_DEBUG build; other builds return SLORA_ERR_INVALID.  Not for
 * serving: the next apply reads the planted value.
 */
int slora_debug_poke_page_table(slora_pool* pool, int64_t entry, int32_t value, int32_t* old);

/*
 * Polls that each of the CUDA-core apply kernel's waits on other warps
 * (stages, v rows, partial sums, the grid barrier) makes before it gives up
 * (0: the built-in limit, 2^24).  A kernel that gives up records
 * SLORA_ERR_TIMEOUT in the device status (slora_device_status), waits with
 * the built-in limit for its own copies still in flight, and returns; y may
 * be partly updated.  For tests of the time-out path.
 */
int slora_debug_set_wait_limit(slora_pool* pool, uint32_t polls);

const char* slora_last_error_string(void);

/*
 * slora_lora_apply_noalloc -- y += s * (x A_a) B_a for one projection,
 * allocating nothing.  The pages describe no counterpart of this entry point.
 *
 * For callers that cannot call cudaMalloc where they compute the delta: a
 * serving runtime that has handed all GPU memory to its own arena (page pool,
 * KV cache, activations) and may not grow its footprint, or code that must
 * not allocate at all while it serves.  Such a caller owns every buffer
 * already; this call needs no slora_pool and makes no cudaMalloc, cudaFree or
 * other allocating call.  Its scratch (token grouping and the fp32 shrink
 * result) is one static device array of SLORA_NOALLOC_SCRATCH_BYTES that
 * every GPU loading the library holds until the process exits.
 *   d_pool, page_elems, dtype   the page pool (device, 16-byte aligned)
 *   d_page_table, pt_stride     device int32; adapter a's entries start at
 *                               a * pt_stride, in the page-table order of
 *                               slora_adapter_load (the layout a pool uses);
 *                               every entry read must name a page of d_pool
 *   d_rank, max_adapters        device int32[max_adapters]; 0 = not resident;
 *                               ranks outside [1, rmax] count as 0, where
 *                               rmax = min(SLORA_MAX_RANK, pt_stride / E) and
 *                               E = sum_q(ceil(in_q/H) + ceil(out_q/H)) is
 *                               the entries one unit of rank takes, so no
 *                               adapter's rows run into the next adapter's
 *                               stretch of the page table
 *   num_proj, proj_in, proj_out host arrays: every projection adapters carry
 *   proj                        the projection to apply
 *   d_token_adapter, T          device int32[T], ids in [-1, max_adapters);
 *                               T <= SLORA_NOALLOC_MAX_TOKENS (else
 *                               SLORA_ERR_INVALID); tokens with id -1 or a
 *                               non-resident adapter are left unchanged
 *   d_x, ldx, d_y, ldy, s       as in slora_lora_apply
 *   stream                      cudaStream_t (NULL = legacy default stream)
 *   status                      optional (NULL: not reported): one int32 in
 *                               device memory or pinned host memory that
 *                               receives this call's device status on
 *                               `stream` once its kernels are done --
 *                               SLORA_OK, SLORA_ERR_NOT_RESIDENT (a token's
 *                               adapter has rank 0), SLORA_ERR_INVALID (an id
 *                               other than -1 outside [0, max_adapters)) or
 *                               SLORA_ERR_TIMEOUT (a kernel's bounded wait
 *                               gave up; y may be partly updated).  Read it
 *                               after synchronising the stream.
 * The first call on a device sets that device up (it looks up the device
 * address of the scratch array and sizes the kernels' grids); make that first
 * call before any stream capture.  Every call shares the one scratch array
 * and leaves the last call's contents in it: calls that may overlap on the
 * GPU (other streams, other threads) race and must be serialised by the
 * caller.
 */
#define SLORA_NOALLOC_MAX_TOKENS 2048
#define SLORA_NOALLOC_SCRATCH_BYTES 2351360u /* 2.24 MiB: grouping of 2048 tokens, 32768 ranks, v */
int slora_lora_apply_noalloc(const void* d_pool, int32_t page_elems, int32_t dtype,
                             const int32_t* d_page_table, int64_t pt_stride, const int32_t* d_rank,
                             int32_t max_adapters, int32_t num_proj, const int32_t* proj_in,
                             const int32_t* proj_out, int32_t proj, const int32_t* d_token_adapter,
                             int32_t T, const void* d_x, int64_t ldx, void* d_y, int64_t ldy, float s,
                             void* stream, int32_t* status);

/*
 * ---- Paged key-value cache ----------------------------------------------
 * The KV half of the unified pool (dongaigc.com summary, section 1 "Unified
 * Paging": KV-cache tensors and adapter weights in the pages of one pool;
 * fatihsoysal.com page, section "vLLM'in PagedAttention Mekanizmasi": a
 * request's tokens in fixed-size blocks found through a table).  A slora_kv
 * is one model's cache over a pool: slora_kv_plan turns a step's request
 * lengths into block-table entries and a slot map, slora_kv_append norms and
 * rotates the new tokens' queries and keys and stores keys and values, and
 * slora_kv_attend lets the new tokens attend over everything stored.
 *
 * A page of page_elems elements holds P = page_elems / (heads_kv * head_dim)
 * whole tokens' K (or V) vectors of one layer: one token where the page is
 * the hidden size and every query head has its own key head, several with
 * shared key heads.  P consecutive positions of a request are a block; in
 * every layer it has one page for K and one for V.  Position t of table row i
 * is token t % P of page table[layer][kv][i][t / P], that is row
 * page * P + t % P of the pool seen as a matrix of heads_kv * head_dim
 * columns.
 *
 * All calls enqueue work on the pool's compute stream, allocate nothing after
 * slora_kv_create, never block the host, and can be captured in a CUDA graph
 * (lengths, rows and pages are read on the device at replay).
 */
typedef struct slora_kv slora_kv; /* opaque, owned by the library */

#define SLORA_KV_MAX_REQUESTS 4096 /* table rows, and requests of one batch */
#define SLORA_KV_MAX_HEAD_DIM 256

typedef struct slora_kv_config {
  int32_t layers;        /* >= 1 */
  int32_t heads_q;       /* query heads, a multiple of heads_kv: heads_q / heads_kv of them share a key head */
  int32_t heads_kv;      /* key (and value) heads */
  int32_t head_dim;      /* a multiple of 16, at most SLORA_KV_MAX_HEAD_DIM */
  int32_t max_requests;  /* rows of the block table, 1 .. SLORA_KV_MAX_REQUESTS */
  int32_t max_blocks;    /* entries of a row: a request holds at most max_blocks * P tokens (<= 2^30) */
} slora_kv_config;

/*
 * The planned batch.  Its arrays lie in the caller's d_arrays (see
 * slora_kv_create), at the same places in every batch: the next slora_kv_plan
 * on the cache overwrites them and makes earlier batches stale.  A batch serves the
 * cache that planned it alone (both by the generation).
 */
typedef struct slora_kv_batch {
  int32_t R;                /* requests */
  int32_t T;                /* tokens the batch has room for */
  int32_t max_new;
  const int32_t* q_start;   /* [R + 1] first token of each request; q_start[R] = tokens in use */
  const int32_t* kv_len;    /* [R] tokens each request holds once the step's are appended; 0: left out */
  const int32_t* tok_req;   /* [T] request of each token, -1: none */
  const int32_t* tok_pos;   /* [T] position of each token in its request, -1: none */
  const int32_t* slots;     /* [layers][2][slot_stride] pool row of each token's K and V, -1: none */
  int64_t slot_stride;      /* the pool's max_tokens */
  uint64_t generation;
} slora_kv_batch;

/*
 * A cache over `pool` (not a planning pool), which must outlive it.  d_table:
 * caller-owned device memory, int32 [layers][2][max_requests][max_blocks],
 * set to -1 here on the compute stream; slora_kv_plan writes the entries of
 * the blocks a step opens.  The caller may write entries too, on the compute
 * stream: a row that starts with another row's entries shares that prefix.
 * page_elems must be a multiple of heads_kv * head_dim.  Batches are of at
 * most the pool's max_tokens tokens.  d_arrays: caller-owned device memory,
 * int32, 16-byte aligned, as many as slora_kv_array_ints says, zeroed here; the
 * batch arrays.
 * Both must outlive the cache.  Allocates the rotary table and the
 * attention's scratch with cudaMalloc.
 */
int slora_kv_array_ints(const slora_pool* pool, const slora_kv_config* config, int64_t* n);
int slora_kv_create(slora_kv** out, slora_pool* pool, const slora_kv_config* config, int32_t* d_table,
                    int32_t* d_arrays);
/* Synchronises the compute stream and frees what slora_kv_create allocated. */
int slora_kv_destroy(slora_kv* kv);

/*
 * Rotary positions for slora_kv_append: the first rot_dim elements of every
 * query and key head (a multiple of 16, at most head_dim; 0: no rotation, the
 * state after create) are rot_dim / 2 pairs, and pair i of a token at
 * position t turns by t * h_inv_freq[i] radians and is multiplied by mscale:
 *     (a, b) -> mscale * (a cos - b sin, a sin + b cos).
 * layout SLORA_ROTARY_HALF: pair i = elements i and i + rot_dim / 2;
 * SLORA_ROTARY_INTERLEAVED: elements 2i and 2i + 1.  h_inv_freq: host, copied
 * before the call returns.  Every scaling of the frequencies for long
 * contexts is a choice of h_inv_freq and mscale.  The turn is reduced as a
 * 64-bit fixed-point fraction of a circle (t times the frequency modulo 2^64),
 * so that what is left of it is the frequency's own error: at most
 * t * h_inv_freq[i] * 2^-55 turn (2^-25 for frequency 1 at position 2^30).  The
 * rest is fp32: the angle within half a turn to 2^-25 turn, its cosine and sine
 * to about 2^-21.
 * Errors: SLORA_ERR_INVALID (sizes, layout, a frequency or mscale that is not
 * finite).  Blocks the host until the compute stream has taken the table;
 * not to be called while the stream is being captured.
 */
#define SLORA_ROTARY_HALF 0
#define SLORA_ROTARY_INTERLEAVED 1
int slora_kv_set_rotary(slora_kv* kv, int32_t rot_dim, int32_t layout, const double* h_inv_freq, float mscale);

/*
 * Plans one step for R requests: request r of table row d_row[r] (NULL: row
 * r; rows of one batch are distinct) holds d_ctx[r] tokens and gets d_new[r]
 * more (0 allowed), whose tokens follow each other in the batch, request by
 * request.  It opens ceil((ctx + new) / P) - ceil(ctx / P) blocks; their
 * pages are taken from d_pages in order, n_pages entries laid out
 * [block][layer][K, V], so one slora_pages_alloc of 2 * layers pages per
 * opened block serves a step as it is.  Entries past the last one needed are
 * not read.  T: the tokens the batch has room for (the rows of q, k, v and
 * out), at least the sum of d_new; a graph captured with a larger T replays
 * smaller batches.  max_new: no request gets more new tokens than this (it
 * picks the kernels slora_kv_attend launches).
 *
 * Arrays are device int32.  What the host cannot check is checked on the GPU
 * and raises the device status SLORA_ERR_INVALID: a row outside the table, a
 * negative length, more new tokens than max_new, or more tokens than a row
 * holds leaves that request out (no tokens, kv_len 0); new tokens beyond T in
 * sum, or blocks beyond d_pages, leave every request out; a page outside the
 * pool becomes entry -1, and its tokens are not stored.
 */
int slora_kv_plan(slora_kv* kv, int32_t R, const int32_t* d_row, const int32_t* d_ctx, const int32_t* d_new,
                  const int32_t* d_pages, int64_t n_pages, int32_t T, int32_t max_new, slora_kv_batch* out);

/*
 * Queries, keys and values of the batch's tokens in one layer.  d_q: T rows
 * of heads_q * head_dim elements, d_k and d_v: T rows of heads_kv * head_dim,
 * row strides ldq, ldk, ldv (so slices of one fused product serve).  With
 * d_q_weight / d_k_weight (head_dim elements each; NULL: no norm) every head
 * x becomes x / sqrt(mean(x^2) + eps) * weight, in fp32; then the rotary turn,
 * in fp32; then one rounding.  Queries go to d_q_out (stride ldqo; may be d_q
 * itself with the same stride, must not overlap it otherwise), keys and
 * values to the tokens' slots; values keep their bits.  Tokens without a
 * request are skipped.  Pointers 16-byte aligned, strides multiples of 8.
 */
int slora_kv_append(slora_kv* kv, const slora_kv_batch* batch, int32_t layer, const void* d_q, int64_t ldq,
                    const void* d_k, int64_t ldk, const void* d_v, int64_t ldv, const void* d_q_weight,
                    const void* d_k_weight, float eps, void* d_q_out, int64_t ldqo);

/*
 * Causal attention of the batch's tokens in one layer over their requests'
 * stored keys and values: for a token at position p, query head h and its key
 * head h / (heads_q / heads_kv),
 *     out = sum_{j <= p} softmax_j(c(scale * q . k_j)) v_j,
 * c(s) = softcap * tanh(s / softcap), or s itself for softcap 0.  The step's
 * own keys and values must be appended first.  scale > 0.  Scores, softmax and sums are
 * fp32 (a sum of n keys' products on the tensor cores may come out n 2^-26 of itself too
 * small), the result is rounded once.  For the product with the values the softmax weights
 * are held in the storage type: in two parts, twice its bits, where a request has at most 8
 * rows (new tokens times query heads of a key head), head_dim is below 64 or above 128, or
 * more than 32 query heads share a key head; elsewhere in one, which adds at most one unit
 * of the type relative to the largest value.  d_q, d_out: T rows of heads_q * head_dim,
 * strides ldq, ldo; out rows of tokens without a request are not written;
 * d_out must not overlap d_q.  Slots past a request's length are never used,
 * whatever they hold; a value that is not finite within a request's stored
 * tokens may reach any of that request's outputs, and no other request's.  A
 * table entry within a request's length that names no page of the pool, K's or
 * V's, raises the device status SLORA_ERR_INVALID, and its tokens are left out
 * of the sums (a row that sees no key at all becomes zeros).
 */
int slora_kv_attend(slora_kv* kv, const slora_kv_batch* batch, int32_t layer, const void* d_q, int64_t ldq,
                    void* d_out, int64_t ldo, float scale, float softcap);

#ifdef __cplusplus
}
#endif
#endif /* SLORA_H */
