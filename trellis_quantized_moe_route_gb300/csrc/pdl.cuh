// Launching: programmatic dependent launches, and the shared memory of large CTAs.
#pragma once

#include <cuda_runtime.h>

#include "per_device.h"

namespace tmoe {

// Programmatic dependent launch: a kernel may start while the one before it in
// the stream still runs; before it touches global memory it waits for that one
// to end, and it lets the next one start as soon as all its own CTAs run.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void grid_launch() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// A launch that may start while the kernel before it ends.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// SMs of the current device.
inline cudaError_t current_sms(int& sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e == cudaSuccess ? cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) : e;
}

// Lets `kern` have `bytes` of dynamic shared memory on the current device. (The
// limit belongs to a device's copy of the kernel; `done`: one for each kernel.)
template <typename... P>
cudaError_t allow_smem(OncePerDevice& done, void (*kern)(P...), int bytes) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return done(dev, [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
}

}  // namespace tmoe
