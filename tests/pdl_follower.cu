// A kernel launched as a programmatic dependent of whatever was launched before it on its
// stream: it starts early, waits as such a kernel has to (griddepcontrol.wait), and copies.
#include <cstdint>
#include <cuda_runtime.h>

__global__ void copy_kernel(const uint4* from, uint4* to, int64_t n) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) to[i] = from[i];
}

// n: 16-byte words of both buffers
extern "C" int follow(const void* from, void* to, int64_t n, void* stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(8);
  cfg.blockDim = dim3(256);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, copy_kernel, static_cast<const uint4*>(from), static_cast<uint4*>(to), n);
}
