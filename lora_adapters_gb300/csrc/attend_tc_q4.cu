// Launches of the chunk kernel (attend_tc.cuh) over caches held in 4 bits.
#include "attend_tc.cuh"

namespace slora {
namespace {

template <class E, int CAP>
void (*chunk_kernel(int head_dim, int groups))(const KvAttendArgs) {
  return head_dim == 128  ? kv_chunk_kernel<E, CAP, 8, 4>
         : head_dim == 64 ? kv_chunk_kernel<E, CAP, 4, 2>
         : groups == 3    ? kv_chunk_kernel<E, CAP, 0, 3>
                          : kv_chunk_kernel<E, CAP, 0, 4>;
}
template <class E>
void (*chunk_kernel(int cap, int head_dim, int groups))(const KvAttendArgs) {
  return cap == kCapNone    ? chunk_kernel<E, kCapNone>(head_dim, groups)
         : cap == kCapSmall ? chunk_kernel<E, kCapSmall>(head_dim, groups)
                            : chunk_kernel<E, kCapAny>(head_dim, groups);
}
void (*chunk_kernel(int dtype, int cap, int head_dim, int groups))(const KvAttendArgs) {
  return dtype == 0 ? chunk_kernel<__half>(cap, head_dim, groups) : chunk_kernel<__nv_bfloat16>(cap, head_dim, groups);
}

}  // namespace

cudaError_t prepare_kv_q4_chunk_kernels(int dtype, int head_dim) {
  for (int cap : {kCapNone, kCapSmall, kCapAny}) {
    const cudaError_t e = cudaFuncSetAttribute(chunk_kernel(dtype, cap, head_dim, (head_dim + 31) / 32),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes<true>);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_kv_q4_chunk(const KvAttendArgs& a, int dtype, int num_sms, cudaStream_t st) {
  const int cap = a.softcap == 0.f ? kCapNone : a.softcap <= kCapNear ? kCapSmall : kCapAny;
  chunk_kernel(dtype, cap, a.kv.head_dim, a.kv.groups)<<<num_sms, kThreads, kSmemBytes<true>, st>>>(a);
  return cudaGetLastError();
}

}  // namespace slora
