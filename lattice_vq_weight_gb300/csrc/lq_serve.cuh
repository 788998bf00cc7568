// Helpers shared by the operators that serve requests from the paged 8-bit KV
// cache (lq_kv_plan.cu, lq_rope.cu, lq_kv_paged.cu, lq_attn_paged.cu,
// lq_verify.cu).  Internal to the library.
#pragma once

#include <climits>
#include <cstdint>

#include <cuda_runtime.h>

#include "lq_host.h"

namespace lq {

// Every kernel of these operators is a programmatic dependent launch: it may
// be scheduled while the kernel before it ends, waits for that grid before its
// first access to global memory, and lets the next kernel be scheduled.  What
// an earlier call may have written (any input of these calls) is read with
// ordinary loads: the read-only path (ld.global.nc) is for data that nothing
// writes while the kernel runs, and here the producer may still be at it when
// the kernel starts; nor does the wait keep such loads behind it.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;"); }

namespace serve {

inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
inline bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

// Tokens per cache block: a power of two, so that a slot splits by shifts.
inline bool valid_block_size(int bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }
inline int log2_of(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

template <typename A>
inline lq_status launch(void (*kernel)(A), unsigned grid, unsigned threads, size_t smem, void* stream, const A& args,
                        unsigned cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args) != cudaSuccess) {
    cudaGetLastError();
    return LQ_ERR_CUDA;
  }
  return check_launch();
}

}  // namespace serve
}  // namespace lq
