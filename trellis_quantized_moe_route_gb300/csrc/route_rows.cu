// Weighted sum of the routes' rows and its gradient (sm_103a).
//   out_t      = sum_j w_tj rows_(t k + j)          in order j = 0..k-1, fp32
//   drows_tk+j = w_tj dout_t,   dw_tj = <dout_t, rows_(t k + j)>
// Rows lie in route order (r = t k + j), as the MXFP4 expert products write
// them. A route of weight zero is left out of the sum, so that a row nobody
// wrote cannot turn 0 into NaN.
#include <algorithm>

#include "elem.cuh"
#include "status.h"

namespace tmoe {

namespace {

constexpr int kCbVec = 8;  // elements of a thread

template <typename T>
__global__ void __launch_bounds__(256) k_combine_routes(const T* __restrict__ rows, const float* __restrict__ w, int T_,
                                                        int k, int H, bool vec, float* __restrict__ out) {
  const int per = (H + kCbVec - 1) / kCbVec;
  const long total = (long)T_ * per;
  for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (long)gridDim.x * blockDim.x) {
    const long t = i / per;
    const int h = (int)(i - t * per) * kCbVec;
    float acc[kCbVec] = {};
    const bool whole = h + kCbVec <= H;
    for (int j = 0; j < k; ++j) {
      const float wj = __ldg(w + t * k + j);
      const T* row = rows + ((size_t)t * k + j) * H + h;
      if (wj == 0.0f) continue;
      if (whole) {
        float v[kCbVec];
        load_f32<kCbVec>(row, vec, v);
#pragma unroll
        for (int x = 0; x < kCbVec; ++x) acc[x] = fmaf(wj, v[x], acc[x]);
      } else {
        for (int x = 0; h + x < H; ++x) acc[x] = fmaf(wj, to_f32(row[x]), acc[x]);
      }
    }
    float* o = out + (size_t)t * H + h;
    if (whole) {
      store_f32<kCbVec>(o, vec, acc);
    } else {
      for (int x = 0; h + x < H; ++x) o[x] = acc[x];
    }
  }
}

constexpr int kCbChunk = 8;  // routes whose dot products a block holds at once

// One block per token.
template <typename T>
__global__ void __launch_bounds__(256) k_combine_routes_bwd(const T* __restrict__ rows, const float* __restrict__ w,
                                                            const float* __restrict__ gout, int T_, int k, int H,
                                                            bool vec, T* __restrict__ grows, float* __restrict__ gw) {
  __shared__ float s_dot[8][kCbChunk];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = blockDim.x >> 5;
  for (int t = blockIdx.x; t < T_; t += gridDim.x) {
    for (int j0 = 0; j0 < k; j0 += kCbChunk) {
      const int nj = min(kCbChunk, k - j0);
      float dot[kCbChunk] = {};
      for (int h = threadIdx.x * kCbVec; h < H; h += blockDim.x * kCbVec) {
        float g[kCbVec];
        const bool whole = h + kCbVec <= H;
        if (whole) {
          load_f32<kCbVec>(gout + (size_t)t * H + h, vec, g);
        } else {
#pragma unroll
          for (int x = 0; x < kCbVec; ++x) g[x] = h + x < H ? gout[(size_t)t * H + h + x] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < kCbChunk; ++j) {
          if (j >= nj) break;
          const size_t r = ((size_t)t * k + j0 + j) * H + h;
          const float wj = w[(size_t)t * k + j0 + j];
          float v[kCbVec];
          if (whole) {
            load_f32<kCbVec>(rows + r, vec, v);
          } else {
#pragma unroll
            for (int x = 0; x < kCbVec; ++x) v[x] = h + x < H ? to_f32(rows[r + x]) : 0.0f;
          }
#pragma unroll
          for (int x = 0; x < kCbVec; ++x) {
            dot[j] = fmaf(g[x], v[x], dot[j]);
            v[x] = wj * g[x];
          }
          if (grows) {
            if (whole) {
              store_f32<kCbVec>(grows + r, vec, v);
            } else {
              for (int x = 0; h + x < H; ++x) grows[r + x] = from_f32<T>(v[x]);
            }
          }
        }
      }
      if (gw) {
#pragma unroll
        for (int j = 0; j < kCbChunk; ++j) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], o);
          if (lane == 0) s_dot[warp][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < nj) {
          float s = 0.0f;
          for (int u = 0; u < warps; ++u) s += s_dot[u][threadIdx.x];
          gw[(size_t)t * k + j0 + threadIdx.x] = s;
        }
        __syncthreads();
      }
    }
  }
}

tm_status combine_check(const void* rows, int32_t dtype, const float* w, int32_t T, int32_t k, int32_t H) {
  if (!dtype_ok(dtype)) return status_fail(TM_EINVAL, "dtype=%d is not a tm_dtype", dtype);
  if (T < 0) return status_fail(TM_EINVAL, "T=%d < 0", T);
  if (k < 1 || k > 32) return status_fail(TM_EINVAL, "k=%d outside 1..32", k);
  if (H < 1) return status_fail(TM_EINVAL, "H=%d must be >= 1", H);
  if (T > 0 && (!rows || !w)) return status_fail(TM_EINVAL, "rows and w must be non-NULL");
  if (((uintptr_t)rows) % dtype_bytes(dtype)) return status_fail(TM_EINVAL, "rows must be aligned to its elements");
  return TM_OK;
}

bool aligned16(const void* p, size_t row_bytes) { return ((uintptr_t)p) % 16 == 0 && row_bytes % 16 == 0; }

}  // namespace

}  // namespace tmoe

using namespace tmoe;

extern "C" {

tm_status trellis_moe_combine_forward(const void* rows, int32_t dtype, const float* w, int32_t T, int32_t k,
                                      int32_t H, float* out, void* stream) {
  set_last_error("");
  const tm_status s = combine_check(rows, dtype, w, T, k, H);
  if (s != TM_OK) return s;
  if (T == 0) return TM_OK;
  if (!out || ((uintptr_t)out) % 4) return status_fail(TM_EINVAL, "out must be non-NULL and 4-byte aligned");
  const bool vec = aligned16(rows, (size_t)H * dtype_bytes(dtype)) && aligned16(out, (size_t)H * 4);
  const long items = (long)T * ((H + kCbVec - 1) / kCbVec);
  const int ctas = (int)std::min<long>(152 * 16, (items + 255) / 256);
  auto go = [&](auto elem) {
    using E = decltype(elem);
    k_combine_routes<E><<<ctas, 256, 0, (cudaStream_t)stream>>>(static_cast<const E*>(rows), w, T, k, H, vec, out);
    return cudaGetLastError();
  };
  const cudaError_t e = TM_BY_DTYPE(dtype, go);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "combine");
}

tm_status trellis_moe_combine_backward(const void* rows, int32_t dtype, const float* w, const float* grad_out,
                                       int32_t T, int32_t k, int32_t H, void* grad_rows, float* grad_w,
                                       void* stream) {
  set_last_error("");
  const tm_status s = combine_check(rows, dtype, w, T, k, H);
  if (s != TM_OK) return s;
  if (T == 0) return TM_OK;
  if (!grad_out || ((uintptr_t)grad_out) % 4)
    return status_fail(TM_EINVAL, "grad_out must be non-NULL and 4-byte aligned");
  if (!grad_rows && !grad_w) return status_fail(TM_EINVAL, "grad_rows and grad_w are both NULL");
  if (((uintptr_t)grad_rows) % dtype_bytes(dtype))
    return status_fail(TM_EINVAL, "grad_rows must be aligned to its elements");
  const size_t row = (size_t)H * dtype_bytes(dtype);
  const bool vec = aligned16(rows, row) && aligned16(grad_out, (size_t)H * 4) && aligned16(grad_rows, row);
  const int ctas = std::min(T, 152 * 16);
  auto go = [&](auto elem) {
    using E = decltype(elem);
    k_combine_routes_bwd<E><<<ctas, 256, 0, (cudaStream_t)stream>>>(static_cast<const E*>(rows), w, grad_out, T, k, H,
                                                                    vec, static_cast<E*>(grad_rows), grad_w);
    return cudaGetLastError();
  };
  const cudaError_t e = TM_BY_DTYPE(dtype, go);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "combine backward");
}

}  // extern "C"
