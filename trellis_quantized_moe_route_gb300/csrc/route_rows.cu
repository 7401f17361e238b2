// Weighted sum of the routes' rows and its gradient (sm_103a).
//   out_t      = sum_j w_tj rows_(t k + j)          in order j = 0..k-1, fp32
//   drows_tk+j = w_tj dout_t,   dw_tj = <dout_t, rows_(t k + j)>
// Rows lie in route order (r = t k + j), as the MXFP4 expert products write
// them. A route of weight zero is left out of the sum, so that a row nobody
// wrote cannot turn 0 into NaN. Bound by memory: 4096 tokens x 8 rows x 5120 bf16
// take 70 us forward (0.42 GB, 6.0 TB/s) and 118 us backward (0.75 GB, 6.4 TB/s).
#include <algorithm>

#include "elem.cuh"
#include "pdl.cuh"
#include "status.h"

namespace tmoe {

namespace {

// A thread takes eight columns of a token; four routes' loads are in flight at
// once.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_combine_routes(const T* __restrict__ rows, const float* __restrict__ w,
                                                        uint32_t total, FastDiv per, int k, int H,
                                                        float* __restrict__ out) {
  grid_wait();
  grid_launch();
  const uint32_t n = blockIdx.x * 256 + threadIdx.x;
  if (n >= total) return;
  const size_t t = per.div(n);
  const int h = (int)(n - (uint32_t)t * per.d) * 8, len = min(8, H - h);
  float acc[8] = {};
  const T* row = rows + t * k * H + h;
  const float* wt = w + t * k;
  for (int j0 = 0; j0 < k; j0 += 4) {
    Eight<T, VEC> e[4];
    float wj[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      e[u].load(row + (size_t)(j0 + u) * H, j0 + u < k ? len : 0);
      wj[u] = j0 + u < k ? __ldg(wt + j0 + u) : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float v[8];
      e[u].to(v);
#pragma unroll
      for (int x = 0; x < 8; ++x) acc[x] = wj[u] != 0.0f ? fmaf(wj[u], v[x], acc[x]) : acc[x];
    }
  }
  Eight<float, VEC> o;
  o.from(acc);
  o.store(out + t * H + h, len);
}

constexpr int kCbChunk = 8;  // routes whose dot products a block holds at once

// One block per token; a thread takes eight columns at a time, the chunk's
// loads all in flight.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512) k_combine_routes_bwd(const T* __restrict__ rows, const float* __restrict__ w,
                                                            const float* __restrict__ gout, int k, int H,
                                                            T* __restrict__ grows, float* __restrict__ gw) {
  __shared__ float s_dot[16][kCbChunk];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const size_t t = blockIdx.x;
  grid_wait();
  grid_launch();
  for (int j0 = 0; j0 < k; j0 += kCbChunk) {
    float dot[kCbChunk] = {}, wj[kCbChunk];
#pragma unroll
    for (int j = 0; j < kCbChunk; ++j) wj[j] = j0 + j < k ? __ldg(w + t * k + j0 + j) : 0.0f;
    for (int h = threadIdx.x * 8; h < H; h += blockDim.x * 8) {
      const int len = min(8, H - h);
      Eight<float, VEC> ge;
      ge.load(gout + t * H + h, len);
      float g[8];
      const size_t base = (t * k + j0) * H + h;
      if (gw) {
        Eight<T, VEC> e[kCbChunk];
#pragma unroll
        for (int j = 0; j < kCbChunk; ++j) e[j].load(rows + base + (size_t)j * H, j0 + j < k ? len : 0);
        ge.to(g);
#pragma unroll
        for (int j = 0; j < kCbChunk; ++j) {
          float v[8];
          e[j].to(v);
#pragma unroll
          for (int x = 0; x < 8; ++x) dot[j] = fmaf(g[x], v[x], dot[j]);
        }
      }
      if (grows) {
        ge.to(g);
#pragma unroll
        for (int j = 0; j < kCbChunk; ++j) {
          float v[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) v[x] = wj[j] * g[x];
          Eight<T, VEC> o;
          o.from(v);
          o.store(grows + base + (size_t)j * H, j0 + j < k ? len : 0);
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
      if (threadIdx.x < kCbChunk && j0 + threadIdx.x < k) {
        float s = 0.0f;
        for (int u = 0; u < warps; ++u) s += s_dot[u][threadIdx.x];
        gw[t * k + j0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}

tm_status combine_check(const void* rows, int32_t dtype, const float* w, int32_t T, int32_t k, int32_t H) {
  if (!dtype_ok(dtype)) return status_fail(TM_EINVAL, "dtype=%d is not a tm_dtype", dtype);
  if (T < 0) return status_fail(TM_EINVAL, "T=%d < 0", T);
  if (k < 1 || k > 32) return status_fail(TM_EINVAL, "k=%d outside 1..32", k);
  if (H < 1) return status_fail(TM_EINVAL, "H=%d must be >= 1", H);
  if (H > 1 << 30) return status_fail(TM_EUNSUPPORTED, "H=%d is more than %d", H, 1 << 30);
  if (T > 0 && (!rows || !w)) return status_fail(TM_EINVAL, "rows and w must be non-NULL");
  if (((uintptr_t)rows) % dtype_bytes(dtype)) return status_fail(TM_EINVAL, "rows must be aligned to its elements");
  return TM_OK;
}

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
  // pieces of at most 2^30 eighths of a row, so that the kernel's items stay in 32 bits
  const int per = (H + 7) / 8, most = (1 << 30) / per;
  auto go = [&](auto elem, auto vec) {
    using E = decltype(elem);
    for (int t = 0; t < T;) {
      const int n = std::min(most, T - t);
      const uint32_t items = (uint32_t)n * per;
      const cudaError_t e = launch_after(k_combine_routes<E, decltype(vec)::value>, dim3((items + 255) / 256), 256, 0,
                                         (cudaStream_t)stream, static_cast<const E*>(rows) + (size_t)t * k * H,
                                         w + (size_t)t * k, items, FastDiv(per), k, H, out + (size_t)t * H);
      if (e != cudaSuccess) return e;
      t += n;  // (at most T: no overflow)
    }
    return cudaSuccess;
  };
  const bool vec = eights(rows, H, H, dtype_bytes(dtype)) && eights(out, H, H, 4);
  const cudaError_t e = TM_BY_DTYPE_VEC(dtype, vec, go);
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
  const int es = dtype_bytes(dtype);
  const bool vec = eights(rows, H, H, es) && eights(grad_out, H, H, 4) && eights(grad_rows, H, H, es);
  // whole warps, as few passes over the columns as 512 threads need, evenly filled
  const int groups = (H + 7) / 8, passes = (groups + 511) / 512;
  const int threads = ((groups + passes - 1) / passes + 31) / 32 * 32;
  auto go = [&](auto elem, auto v) {
    using E = decltype(elem);
    return launch_after(k_combine_routes_bwd<E, decltype(v)::value>, dim3(T), threads, 0, (cudaStream_t)stream,
                           static_cast<const E*>(rows), w, grad_out, k, H, static_cast<E*>(grad_rows), grad_w);
  };
  const cudaError_t e = TM_BY_DTYPE_VEC(dtype, vec, go);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "combine backward");
}

}  // extern "C"
