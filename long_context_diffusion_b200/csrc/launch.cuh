// Kernel launches with programmatic dependent launch (PDL).
//
// Every kernel of the library is launched with programmatic stream
// serialisation: it may be scheduled while the kernel before it on the stream
// is still finishing, so that launch latency and prologues (barrier set-up,
// tensor-memory allocation, tensor-map prefetch) overlap the predecessor's
// tail.  Each kernel calls pdl_wait() before it reads or writes global memory
// that earlier work on the stream writes or reads (the wait returns once the
// predecessor grid has completed and its writes are visible; without a
// programmatic predecessor it returns at once), and pdl_trigger() once its
// successor may be scheduled.  A successor is scheduled only after every CTA
// of this grid has triggered or exited, i.e. after all of them are resident,
// so an early successor never takes resources this grid still needs; kernels
// that allocate tensor memory trigger only after their allocation.
// Measured inside a CUDA graph of the denoising step, PDL gave no gain (the
// graph's launch gaps are already small), so it is opt-in: the DL_FLAG_PDL
// kernel flag (dl_set_kernel_flags) turns it on; otherwise kernels launch
// plainly and pdl_wait() returns at once.
// The token-by-token calls (dl_qk_norm_rope, dl_decode_attn, dl_evict_select,
// dl_cache_compact) always use it: they run for 4 to 20 us, of which it hides
// 1.5 to 2 (back to back, eager: norm + rotation of a block 6.2 -> 4.8 us, tiny
// attention 8.2 -> 6.4, eviction plan 8.9 -> 6.8, 64 moves 6.2 -> 3.9).  Every
// CTA of their kernels reaches pdl_wait(), so that a grid's completion implies its
// predecessors', and none reads device memory before it: a predecessor that has
// triggered says nothing of the writes of the kernels before it.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <utility>

#include "../../include/dl.h"

namespace dl {

unsigned kernel_flags();  // api.cu

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

inline bool pdl_enabled() { return (kernel_flags() & DL_FLAG_PDL) != 0; }

// `dependent`: programmatic even without the flag.
template <typename... KArgs, typename... Args>
cudaError_t launch_as(bool dependent, void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                      cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent || pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                   Args&&... args) {
  return launch_as(false, kernel, grid, block, smem, st, std::forward<Args>(args)...);
}

// Allows `bytes` of dynamic shared memory to a kernel, once per device.
template <auto Kernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace dl

// Launches and returns the launch error from the enclosing function.
#define DL_LAUNCH_DEPENDENT(...)                              \
  do {                                                        \
    cudaError_t dl_le_ = ::dl::launch_as(true, __VA_ARGS__);  \
    if (dl_le_ != cudaSuccess) return dl_le_;                 \
  } while (0)
#define DL_LAUNCH(...)                                   \
  do {                                                   \
    cudaError_t dl_le_ = ::dl::launch(__VA_ARGS__);      \
    if (dl_le_ != cudaSuccess) return dl_le_;            \
  } while (0)
