// MXFP4 quantisation of rows and its inverse (sm_103a).
//
// codes: 16 bytes a block (value 2i in the low half of byte i), blocks of a row
// in order; scales: one byte a block. A row of K values has ceil(K / 32)
// blocks, the last one filled up with zeros. Bound by memory: a value's s
// bytes are read and 17/32 of a byte written (the inverse the other way).
// 163840 x 1536 bf16: 104 us = 6.1 TB/s and 91 us = 7.0 TB/s.
#include <algorithm>

#include "elem.cuh"
#include "mxfp4.cuh"
#include "pdl.cuh"
#include "status.h"

namespace tmoe {

namespace {

// Four lanes take a block, eight values each: the block's maximum is two
// shuffles away, and a warp reads eight blocks (512 or 1024 bytes) in one or
// two loads of 16 bytes a lane. A CTA takes kQuTile such eighths, four of a
// thread in flight at once: loads behind a branch are converted inside it, one
// waiting for the other, and with those, a 64-bit division a tile and an
// indexed array in local memory the two kernels took 193 and 187 us on 163840 x
// 1536 bf16. The row of an eighth comes from one multiplication.
constexpr int kQuUnroll = 4;
constexpr int kQuTile = 256 * kQuUnroll;

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_mxfp4_quantize(const T* __restrict__ x, int64_t ld, uint32_t total, FastDiv per,
                                                        int K, uint32_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales) {
  grid_wait();
  grid_launch();
  const uint32_t tile = blockIdx.x * kQuTile + threadIdx.x;
  Eight<T, VEC> e[kQuUnroll];
#pragma unroll
  for (int u = 0; u < kQuUnroll; ++u) {
    const uint32_t i = tile + u * 256, r = per.div(i);
    const int col = (int)(i - r * per.d) * 8;
    e[u].load(x + (int64_t)r * ld + col, i < total ? max(0, min(8, K - col)) : 0);
  }
#pragma unroll
  for (int u = 0; u < kQuUnroll; ++u) {
    const uint32_t i = tile + u * 256;
    float v[8];
    e[u].to(v);
    uint32_t byte;
    const uint32_t q = mxfp4_codes(v, e[u].block_amax_bits(), byte);
    if (i < total) {
      codes[i] = q;
      if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_mxfp4_dequantize(const uint32_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, uint32_t total,
                                                          FastDiv per, int K, T* __restrict__ out) {
  grid_wait();
  grid_launch();
  const uint32_t tile = blockIdx.x * kQuTile + threadIdx.x;
  uint32_t c[kQuUnroll], b[kQuUnroll];
#pragma unroll
  for (int u = 0; u < kQuUnroll; ++u) {
    const uint32_t i = tile + u * 256;
    c[u] = i < total ? __ldg(codes + i) : 0u;
    b[u] = i < total ? __ldg(scales + (i >> 2)) : 0u;
  }
#pragma unroll
  for (int u = 0; u < kQuUnroll; ++u) {
    const uint32_t i = tile + u * 256, r = per.div(i);
    const int col = (int)(i - r * per.d) * 8;
    float v[8];
    e2m1x8_to_f32(c[u], v);
    const float s = mxfp4_power(b[u]);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= s;
    Eight<T, VEC> e;
    e.from(v);
    e.store(out + (int64_t)r * K + col, i < total ? max(0, min(8, K - col)) : 0);
  }
}

// Calls f(first row, rows) over pieces of less than 2^30 eighths each, so that
// the kernels' indexes stay in 32 bits.
template <typename F>
cudaError_t by_rows(long rows, int per, F f) {
  const long most = std::max(1L, (1L << 30) / per);
  for (long r = 0; r < rows; r += most) {
    const cudaError_t e = f(r, std::min(most, rows - r));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

unsigned quant_ctas(uint32_t items) { return (items + kQuTile - 1) / kQuTile; }

cudaError_t mxfp4_quantize(const void* x, int dtype, int64_t ld, long rows, int K, uint8_t* codes, uint8_t* scales,
                           cudaStream_t st) {
  const int es = dtype_bytes(dtype), nb = (K + 31) / 32, per = nb * 4;
  auto go = [&](auto elem, auto vec) {
    using T = decltype(elem);
    return by_rows(rows, per, [&](long r, long n) {
      const uint32_t total = (uint32_t)(n * per);
      return launch_after(k_mxfp4_quantize<T, decltype(vec)::value>, dim3(quant_ctas(total)), 256, 0, st,
                             static_cast<const T*>(x) + r * ld, ld, total, FastDiv(per), K,
                             reinterpret_cast<uint32_t*>(codes) + r * per, scales + r * nb);
    });
  };
  return TM_BY_DTYPE_VEC(dtype, eights(x, ld, K, es), go);
}

cudaError_t mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, long rows, int K, void* out, int dtype,
                             cudaStream_t st) {
  const int es = dtype_bytes(dtype), nb = (K + 31) / 32, per = nb * 4;
  auto go = [&](auto elem, auto vec) {
    using T = decltype(elem);
    return by_rows(rows, per, [&](long r, long n) {
      const uint32_t total = (uint32_t)(n * per);
      return launch_after(k_mxfp4_dequantize<T, decltype(vec)::value>, dim3(quant_ctas(total)), 256, 0, st,
                             reinterpret_cast<const uint32_t*>(codes) + r * per, scales + r * nb, total, FastDiv(per), K,
                             static_cast<T*>(out) + r * K);
    });
  };
  return TM_BY_DTYPE_VEC(dtype, eights(out, K, K, es), go);
}

}  // namespace

}  // namespace tmoe

using namespace tmoe;

extern "C" {

tm_status trellis_moe_mxfp4_quantize(const void* x, int32_t dtype, int64_t ld, int64_t rows, int32_t K,
                                     uint8_t* codes, uint8_t* scales, void* stream) {
  set_last_error("");
  if (!dtype_ok(dtype)) return status_fail(TM_EINVAL, "dtype=%d is not a tm_dtype", dtype);
  if (rows < 0) return status_fail(TM_EINVAL, "rows=%lld < 0", (long long)rows);
  if (K < 1 || K > (1 << 30)) return status_fail(TM_EINVAL, "K=%d outside 1..%d", K, 1 << 30);
  if (ld < K) return status_fail(TM_EINVAL, "ld=%lld is less than K=%d", (long long)ld, K);
  if (rows == 0) return TM_OK;
  if (!x || !codes || !scales) return status_fail(TM_EINVAL, "x, codes and scales must be non-NULL");
  if (((uintptr_t)x) % dtype_bytes(dtype)) return status_fail(TM_EINVAL, "x must be aligned to its elements");
  if (((uintptr_t)codes) % 16) return status_fail(TM_EINVAL, "codes must be 16-byte aligned");
  const cudaError_t e = mxfp4_quantize(x, dtype, ld, (long)rows, K, codes, scales, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "MXFP4 quantise");
}

tm_status trellis_moe_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t K,
                                       void* out, int32_t dtype, void* stream) {
  set_last_error("");
  if (!dtype_ok(dtype)) return status_fail(TM_EINVAL, "dtype=%d is not a tm_dtype", dtype);
  if (rows < 0) return status_fail(TM_EINVAL, "rows=%lld < 0", (long long)rows);
  if (K < 1 || K > (1 << 30)) return status_fail(TM_EINVAL, "K=%d outside 1..%d", K, 1 << 30);
  if (rows == 0) return TM_OK;
  if (!codes || !scales || !out) return status_fail(TM_EINVAL, "codes, scales and out must be non-NULL");
  if (((uintptr_t)codes) % 16) return status_fail(TM_EINVAL, "codes must be 16-byte aligned");
  if (((uintptr_t)out) % dtype_bytes(dtype)) return status_fail(TM_EINVAL, "out must be aligned to its elements");
  const cudaError_t e = mxfp4_dequantize(codes, scales, (long)rows, K, out, dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "MXFP4 dequantise");
}

}  // extern "C"
