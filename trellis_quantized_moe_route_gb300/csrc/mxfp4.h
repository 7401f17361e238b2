// Internal launchers of the MXFP4 kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace tmoe {

// rows of x (stride ld elements) -> codes and scales in row order.
cudaError_t launch_mxfp4_quantize(const void* x, int dtype, int64_t ld, long rows, int K, uint8_t* codes,
                                  uint8_t* scales, cudaStream_t st);

}  // namespace tmoe
