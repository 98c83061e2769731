// Launches of the chunk kernel (attend_tc.cuh) over 16-bit caches.
#include "attend_tc.cuh"

namespace slora {
namespace {

template <class E, int CAP>
void (*chunk_kernel(int head_dim))(const KvAttendArgs) {
  return head_dim == 128 ? kv_chunk_kernel<E, CAP, 8, 0> : head_dim == 64 ? kv_chunk_kernel<E, CAP, 4, 0>
                                                                       : kv_chunk_kernel<E, CAP, 0, 0>;
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
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes<false>);
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

int64_t kv_chunk_part_rows(int num_sms) { return (int64_t)num_sms * 4 * kKvTile; }

cudaError_t launch_kv_chunk(const KvAttendArgs& a, int dtype, int num_sms, cudaStream_t st) {
  const int cap = a.softcap == 0.f ? kCapNone : a.softcap <= kCapNear ? kCapSmall : kCapAny;
  chunk_kernel(dtype, cap, a.kv.head_dim)<<<num_sms, kThreads, kSmemBytes<false>, st>>>(a);
  return cudaGetLastError();
}

}  // namespace slora
