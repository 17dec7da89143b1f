// What the small kernels beside the 16-bit products share: their launch and pieces of eight elements.
#pragma once

#include "mm16.cuh"

namespace ds4 {
namespace {

// Programmatic dependent launch, as in the products: a kernel sets itself up while its predecessor runs, and touches
// global memory only after that is complete.
__device__ __forceinline__ void begin() {
  asm volatile("griddepcontrol.wait;\n griddepcontrol.launch_dependents;\n" ::: "memory");
}
template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Eight 16-bit elements that are also moved as one 16-byte piece (a plain array is aligned to 2 bytes only, and the piece's
// loads and stores could fault wherever the compiler keeps it in memory).
struct Eight {
  alignas(16) uint16_t h[8];
  __device__ __forceinline__ uint4& piece() { return *reinterpret_cast<uint4*>(h); }
};
static_assert(alignof(Eight) >= alignof(uint4) && sizeof(Eight) == sizeof(uint4), "a piece of eight elements");

}  // namespace
}  // namespace ds4
