// Pieces of the decode kernels of slora_kv_attend: loads, warp-level products, the
// cut of the work into runs (attend.cu: 16-bit caches, attend_q4.cu: caches in 4 bits).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "kv.cuh"
#include "kv.h"

namespace slora {

constexpr int kDecMinUnits = 1;          // shortest run (one 640-token request: 12.5 us with 1, 13.0 with 2, 15.6 with 4)

// Streaming 16-byte load: every byte of the cache is used once per call, and the
// rest of its 256 bytes by the same warp or its neighbours (1 % on 7B decode).
__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
template <class E>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (Elem<E>::kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8x8 matrix of 16-bit elements held as one packed pair a lane.
__device__ __forceinline__ uint32_t trans8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The units of a call: segment = (request, row tile of kKvRowTile rows, block
// of `hbw` key heads), ceil(len / kv.unit) units each, laid out request by request.
struct DecSplit {
  int64_t total;     // units
  int64_t run;       // units per group of warps
};
__device__ __forceinline__ DecSplit dec_split(int units, int blocks, int64_t groups) {
  DecSplit s;
  s.total = (int64_t)units * blocks;
  s.run = max((int64_t)kDecMinUnits, (s.total + groups - 1) / groups);
  return s;
}
// Largest r with off[r] * blocks <= x, by a whole warp: the lanes look at 32
// places of what is left at a time.
__device__ __forceinline__ int find_request(const int32_t* off, int R, int64_t x, int blocks) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = R;               // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5, i = lane * step;
    const bool le = i < n && (int64_t)__ldg(off + lo + i) * blocks <= x;
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);   // off[lo] <= x always
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

// The largest power of two up to 16 that divides the key heads.
inline int heads_abreast(int heads_kv) {
  int n = 1;
  while (n < 16 && heads_kv % (2 * n) == 0) n *= 2;
  return n;
}

// A launch that may begin before the one ahead of it in the stream has ended.
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace slora
