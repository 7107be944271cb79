// Launches that overlap the end of the kernel before them.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"

namespace dprc {

// Launches `kernel` so that it may start while the kernel before it in the
// stream ends; the kernel waits for that one (pdl_wait) before it reads or
// writes anything.  A tensor-core map of 16384 x 1024 x 1024 bf16 takes 32 us
// back to back where it takes 37 us behind the full end of the kernel before.
// What such a kernel reads may be written while it lives, so that it reads by
// coherent loads only: never __ldg, ld.global.nc, or a plain read of what a
// const __restrict__ parameter points to, which the compiler may turn into one.
// cl: CTAs per cluster.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, int cl, cudaStream_t s,
                         size_t smem, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cl;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Allows a kernel its shared memory, once per device.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
  constexpr int kMaxDev = 64;
  static std::atomic<int> done[kMaxDev];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kMaxDev;
  if (known && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && known) done[dev].store(1, std::memory_order_release);
  return e;
}

// Loads of such a kernel with a cache policy: coherent, and volatile, so that the
// compiler leaves each behind the kernel's wait.  ld_l2: from L2, not kept in L1;
// ld_stream: to be evicted first; ld_once: a coherent load that leaves L1 as it is.
#define DPRC_LOAD(name, op)                                                                 \
  template <typename T>                                                                     \
  __device__ __forceinline__ T name(const T* p) {                                           \
    static_assert(sizeof(T) == 2 || sizeof(T) == 4 || sizeof(T) == 8 || sizeof(T) == 16,    \
                  "one access");                                                            \
    T r;                                                                                    \
    if constexpr (sizeof(T) == 2) {                                                         \
      asm volatile("ld.global" op ".b16 %0, [%1];"                                          \
                   : "=h"(*reinterpret_cast<unsigned short*>(&r))                           \
                   : "l"(p));                                                               \
    } else if constexpr (sizeof(T) == 4) {                                                  \
      asm volatile("ld.global" op ".b32 %0, [%1];"                                          \
                   : "=r"(*reinterpret_cast<uint32_t*>(&r))                                 \
                   : "l"(p));                                                               \
    } else if constexpr (sizeof(T) == 8) {                                                  \
      asm volatile("ld.global" op ".b64 %0, [%1];"                                          \
                   : "=l"(*reinterpret_cast<unsigned long long*>(&r))                       \
                   : "l"(p));                                                               \
    } else {                                                                                \
      uint32_t* u = reinterpret_cast<uint32_t*>(&r);                                        \
      asm volatile("ld.global" op ".v4.b32 {%0, %1, %2, %3}, [%4];"                         \
                   : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])                         \
                   : "l"(p));                                                               \
    }                                                                                       \
    return r;                                                                               \
  }
DPRC_LOAD(ld_l2, ".cg")
DPRC_LOAD(ld_stream, ".cs")
DPRC_LOAD(ld_once, ".L1::no_allocate")
#undef DPRC_LOAD

// The two ends of a kernel that may run beside the one before it (launch_after).
// It may where nothing it reads or writes is that kernel's, and that kernel let
// it start only after its own wait (as beside_begin does), so that everything
// before that kernel is complete.  The wait that is left out at the start comes
// at the end: the next kernel's wait then covers both.
__device__ __forceinline__ void beside_begin(bool beside) {
  if (!beside) pdl_wait();
  pdl_launch_dependents();
}
__device__ __forceinline__ void beside_end(bool beside) {
  if (beside && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) pdl_wait();
}

}  // namespace dprc
