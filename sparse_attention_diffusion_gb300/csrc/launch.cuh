// Launches whose start overlaps the end of the kernel before them in the stream
// (programmatic dependent launch). Such a kernel may be on the SMs before its
// predecessor has finished: every thread of it calls grid_inputs_ready() before
// its first access to global memory, which waits until the predecessor is done
// and its writes are visible, and then grid_let_next_start(). The second call
// comes after the first and after any tensor-memory allocation, so that a waiting
// successor can never hold what a running kernel still needs.
//
// The second kernel of a pair that one call launches directly behind each other may read what the call was given (not what the
// first kernel makes) before it waits: the first one lets it start only after its own wait, so everything that the call follows
// is done by then. This holds as long as (1) nothing is launched between the two, (2) every thread of the first that lets
// the second start has waited before, and (3) some thread of every block of the second waits before the block ends, so that
// whatever follows the second, which may overwrite the workspace, finds both done. Three kernels do so: packed_join_kernel (the
// bounds of the sequences), linear_pair_kernel and linear_few_kernel with adapters (x and w).
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"

namespace mcs {

__device__ __forceinline__ void grid_inputs_ready() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Lets a kernel use `bytes` of dynamic shared memory, once per device (bytes must
// be the same in every call for one kernel; plans that differ share the kernel's
// attribute between threads).
template <auto kKern>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};  // one bit per device, of this kernel
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kKern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// allow_smem for a kernel that moves registers between its warps, which must have been compiled with as many as
// it counts on.
template <auto kKern>
cudaError_t allow_smem_and_regs(int bytes, int regs) {
  static std::atomic<bool> checked{false};
  if (!checked.load(std::memory_order_relaxed)) {
    cudaFuncAttributes fa{};
    const cudaError_t e = cudaFuncGetAttributes(&fa, kKern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < regs) return cudaErrorInvalidConfiguration;
    checked.store(true, std::memory_order_relaxed);
  }
  return allow_smem<kKern>(bytes);
}

// cluster: CTAs of a cluster along x (0: the kernel's own attribute, or none).
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kern)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s, unsigned cluster,
                              Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 0) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, Params(args)...);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace mcs
