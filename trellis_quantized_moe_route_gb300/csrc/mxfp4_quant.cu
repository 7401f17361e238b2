// MXFP4 quantisation of rows and its inverse (sm_103a).
//
// codes: 16 bytes a block (value 2i in the low half of byte i), blocks of a row
// in order; scales: one byte a block. A row of K values has ceil(K / 32)
// blocks, the last one filled up with zeros. Bound by memory: a value's s
// bytes are read and 17/32 of a byte written (the inverse the other way).
#include <algorithm>

#include "elem.cuh"
#include "mxfp4.cuh"
#include "status.h"

namespace tmoe {

namespace {

// Four lanes take a block, eight values each: the block's maximum is two
// shuffles away, and a warp reads eight blocks (512 or 1024 bytes) in one or
// two loads of 16 bytes a lane.
template <typename T>
__global__ void __launch_bounds__(256) k_mxfp4_quantize(const T* __restrict__ x, int64_t ld, long rows, int K, bool vec,
                                                        uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int nb = (K + 31) / 32;
  const long total = rows * nb * 4;
  const long stride = (long)gridDim.x * blockDim.x;
  const long padded = (total + 31) / 32 * 32;  // whole warps take part in the shuffles
  for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < padded; i += stride) {
    float v[8];
    const long blk = i >> 2;
    const long row = blk / nb;
    const int col = (int)(blk - row * nb) * 32 + (int)(i & 3) * 8;
    const T* p = x + row * ld + col;
    if (i < total && col + 8 <= K) {
      load_f32<8>(p, vec, v);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = i < total && col + c < K ? to_f32(p[c]) : 0.0f;
    }
    uint32_t m = 0;  // |v| as bits: ordered like the values, a NaN above every number
#pragma unroll
    for (int c = 0; c < 8; ++c) m = max(m, __float_as_uint(v[c]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const uint32_t byte = mxfp4_scale_byte(m);
    const float inv = mxfp4_inverse(byte);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] *= inv;
    const uint32_t q = byte == 255u ? 0u : e2m1x8(v);
    if (i < total) {
      codes[i] = q;
      if ((i & 3) == 0) scales[blk] = (uint8_t)byte;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) k_mxfp4_dequantize(const uint32_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, long rows, int K,
                                                          bool vec, T* __restrict__ out) {
  const int nb = (K + 31) / 32;
  const long total = rows * nb * 4;
  for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (long)gridDim.x * blockDim.x) {
    const long blk = i >> 2;
    const long row = blk / nb;
    const int col = (int)(blk - row * nb) * 32 + (int)(i & 3) * 8;
    float v[8];
    e2m1x8_to_f32(__ldg(codes + i), v);
    const float s = mxfp4_power(__ldg(scales + blk));
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] *= s;
    T* o = out + row * K + col;
    if (col + 8 <= K) {
      store_f32<8>(o, vec, v);
    } else {
      for (int c = 0; col + c < K; ++c) o[c] = from_f32<T>(v[c]);
    }
  }
}

int quant_ctas(long items) { return (int)std::min<long>(152 * 16, (items + 255) / 256); }

}  // namespace

cudaError_t launch_mxfp4_quantize(const void* x, int dtype, int64_t ld, long rows, int K, uint8_t* codes,
                                  uint8_t* scales, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int es = dtype_bytes(dtype);
  const bool vec = ((uintptr_t)x) % 16 == 0 && (ld * es) % 16 == 0;
  auto go = [&](auto elem) {
    using T = decltype(elem);
    k_mxfp4_quantize<T><<<quant_ctas(rows * ((K + 31) / 32) * 4), 256, 0, st>>>(
        static_cast<const T*>(x), ld, rows, K, vec, reinterpret_cast<uint32_t*>(codes), scales);
    return cudaGetLastError();
  };
  return TM_BY_DTYPE(dtype, go);
}

}  // namespace tmoe

using namespace tmoe;

extern "C" {

tm_status trellis_moe_mxfp4_quantize(const void* x, int32_t dtype, int64_t ld, int64_t rows, int32_t K,
                                     uint8_t* codes, uint8_t* scales, void* stream) {
  set_last_error("");
  if (!dtype_ok(dtype)) return status_fail(TM_EINVAL, "dtype=%d is not a tm_dtype", dtype);
  if (rows < 0) return status_fail(TM_EINVAL, "rows=%lld < 0", (long long)rows);
  if (K < 1) return status_fail(TM_EINVAL, "K=%d must be >= 1", K);
  if (ld < K) return status_fail(TM_EINVAL, "ld=%lld is less than K=%d", (long long)ld, K);
  if (rows == 0) return TM_OK;
  if (!x || !codes || !scales) return status_fail(TM_EINVAL, "x, codes and scales must be non-NULL");
  if (((uintptr_t)x) % dtype_bytes(dtype)) return status_fail(TM_EINVAL, "x must be aligned to its elements");
  if (((uintptr_t)codes) % 16) return status_fail(TM_EINVAL, "codes must be 16-byte aligned");
  const cudaError_t e = launch_mxfp4_quantize(x, dtype, ld, (long)rows, K, codes, scales, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "MXFP4 quantise");
}

tm_status trellis_moe_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t K,
                                       void* out, int32_t dtype, void* stream) {
  set_last_error("");
  if (!dtype_ok(dtype)) return status_fail(TM_EINVAL, "dtype=%d is not a tm_dtype", dtype);
  if (rows < 0) return status_fail(TM_EINVAL, "rows=%lld < 0", (long long)rows);
  if (K < 1) return status_fail(TM_EINVAL, "K=%d must be >= 1", K);
  if (rows == 0) return TM_OK;
  if (!codes || !scales || !out) return status_fail(TM_EINVAL, "codes, scales and out must be non-NULL");
  if (((uintptr_t)codes) % 16) return status_fail(TM_EINVAL, "codes must be 16-byte aligned");
  const int es = dtype_bytes(dtype);
  if (((uintptr_t)out) % es) return status_fail(TM_EINVAL, "out must be aligned to its elements");
  const bool vec = ((uintptr_t)out) % 16 == 0 && ((size_t)K * es) % 16 == 0;
  auto go = [&](auto elem) {
    using T = decltype(elem);
    k_mxfp4_dequantize<T><<<quant_ctas(rows * ((K + 31) / 32) * 4), 256, 0, (cudaStream_t)stream>>>(
        reinterpret_cast<const uint32_t*>(codes), scales, (long)rows, K, vec, static_cast<T*>(out));
    return cudaGetLastError();
  };
  const cudaError_t e = TM_BY_DTYPE(dtype, go);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "MXFP4 dequantise");
}

}  // extern "C"
