// Launches whose set-up overlaps the end of the kernel before them in the
// stream (programmatic stream serialization).
//
// A kernel launched this way calls grid_dependency_wait() before it reads or
// writes anything in global memory (it may ask for data as far as L2, where all
// writes meet); that returns once every kernel it follows has
// finished and its writes are visible, so the order of results is that of an
// ordinary launch.  (What other kernels write is read with plain or L2 loads:
// the read-only path assumes data that does not change while the kernel runs,
// its time before the wait included.)  grid_dependency_trigger() lets the next such kernel start
// its own set-up; it comes where a block needs nothing more that a waiting
// block could hold (its tensor memory is allocated, its loads are issued).
// One token through a linear layer, calls back to back: 12.8 us, 14.5 without.  Small
// norms and quantisers trigger right after their own wait (a layer's four kernels
// on one token: 28.1 us, 30.0 without).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <utility>

namespace forge {

__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// A number above 0 that a launch works out once per device (attributes set, CTAs
// that fit).  Threads whose first calls meet may both work it out.
class PerDevice {
 public:
  // make(&n) answers with an error or sets n.
  template <typename F>
  cudaError_t get(int* n, F&& make) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool kept = dev >= 0 && dev < kMax;
    *n = kept ? value_[dev].load(std::memory_order_acquire) : 0;
    if (*n > 0) return cudaSuccess;
    e = make(n);
    if (e == cudaSuccess && kept) value_[dev].store(*n, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kMax = 64;
  std::atomic<int> value_[kMax] = {};
};
// The launches of `kern` may use `bytes` of dynamic shared memory.
template <typename Kern>
cudaError_t allow_smem(PerDevice& once, Kern kern, int bytes) {
  int n = 0;
  return once.get(&n, [&](int* v) {
    *v = 1;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
}

// cluster_x: CTAs per cluster (0: no clusters).  A launch that fails answers with
// its error and leaves none behind for the check after another launch.
template <typename... P, typename... A>
cudaError_t launch_chained_2d(void (*kern)(P...), dim3 grid, unsigned block, size_t smem,
                              unsigned cluster_x, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(block, 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster_x;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = cluster_x > 0 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&lc, kern, std::forward<A>(args)...);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kern)(P...), unsigned grid, unsigned block, size_t smem,
                           unsigned cluster_x, cudaStream_t stream, A&&... args) {
  return launch_chained_2d(kern, dim3(grid, 1, 1), block, smem, cluster_x, stream,
                           std::forward<A>(args)...);
}

}  // namespace forge
