// Products with MXFP4 weights (sm_103a): y = deq(q(x)) deq(W)^T for a dense
// matrix or for each route's expert, with the rows of x quantised to MXFP4 in
// the call. A product of two codes is a multiple of 1/4 of at most 36, so a
// block's 32 products add up exactly in fp32; the blocks' sums, each times its
// two powers of two, are added in fp32.
#include <algorithm>
#include <new>

#include "elem.cuh"
#include "mxfp4.h"
#include "mxfp4.cuh"
#include "status.h"

struct tm_mxfp4 {
  tm_mxfp4_desc desc;
};

namespace tmoe {

namespace {

constexpr size_t kMxAlign = 256;
size_t mx_align(size_t v) { return (v + kMxAlign - 1) / kMxAlign * kMxAlign; }
int mx_blocks(int K) { return (K + 31) / 32; }

// Error word | codes of x | scales of x
struct MxLayout {
  size_t codes, scales, total;
};

MxLayout mx_layout(const tm_mxfp4_desc& d, long rows) {
  MxLayout L;
  L.codes = kMxAlign;
  L.scales = L.codes + mx_align((size_t)rows * mx_blocks(d.K) * 16);
  L.total = L.scales + mx_align((size_t)rows * mx_blocks(d.K));
  return L;
}

// One warp: one row of y, 32 output channels (one a lane).
template <typename T>
__global__ void __launch_bounds__(128) k_mx_rows(const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
                                                 const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
                                                 const int32_t* __restrict__ ids, int rows, int x_div, int E, int N,
                                                 int nb, int gated, T* __restrict__ out, uint32_t* __restrict__ err) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.y * 4 + warp;
  const int n = blockIdx.x * 32 + lane;
  if (r >= rows || n >= N) return;
  const int e = ids ? ids[r] : 0;
  if (e < 0 || e >= E) {
    if (n == 0) atomicOr(err, 1u);
    out[(size_t)r * N + n] = from_f32<T>(0.0f);
    return;
  }
  const size_t xr = (size_t)(r / x_div) * nb;
  const size_t wr0 = ((size_t)e * (gated ? 2 * N : N) + n) * nb;
  float y[2] = {0.0f, 0.0f};
  for (int half = 0; half <= gated; ++half) {
    const size_t wr = wr0 + (size_t)half * N * nb;
    float acc = 0.0f;
    for (int b = 0; b < nb; ++b) {
      float s = 0.0f;
      for (int c = 0; c < 4; ++c) {
        float a[8], w[8];
        e2m1x8_to_f32(__ldg(reinterpret_cast<const uint32_t*>(xc) + (xr + b) * 4 + c), a);
        e2m1x8_to_f32(__ldg(reinterpret_cast<const uint32_t*>(wc) + (wr + b) * 4 + c), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(a[i], w[i], s);
      }
      acc += s * mxfp4_power(xs[xr + b]) * mxfp4_power(ws[wr + b]);
    }
    y[half] = acc;
  }
  const float v = gated ? y[0] / (1.0f + expf(-y[0])) * y[1] : y[0];
  out[(size_t)r * N + n] = from_f32<T>(v);
}

__global__ void k_mx_clear(uint32_t* err) { *err = 0; }

struct MxCall {
  const void* x;
  int x_dtype;
  int64_t ld;
  const int32_t* ids;
  int rows;    // rows of y
  int x_rows;
  int x_div;   // row r of y reads row r / x_div of x
  void* out;
  int out_dtype;
  void* ws;
};

cudaError_t mx_run(const tm_mxfp4_desc& d, const MxCall& c, cudaStream_t st) {
  const MxLayout L = mx_layout(d, c.rows);
  uint8_t* base = static_cast<uint8_t*>(c.ws);
  uint32_t* err = reinterpret_cast<uint32_t*>(base);
  k_mx_clear<<<1, 1, 0, st>>>(err);
  cudaError_t e = launch_mxfp4_quantize(c.x, c.x_dtype, c.ld, c.x_rows, d.K, base + L.codes, base + L.scales, st);
  if (e != cudaSuccess) return e;
  auto go = [&](auto elem) {
    using T = decltype(elem);
    k_mx_rows<T><<<dim3((d.N + 31) / 32, (c.rows + 3) / 4), 128, 0, st>>>(
        base + L.codes, base + L.scales, d.codes, d.scales, c.ids, c.rows, c.x_div, d.E, d.N, mx_blocks(d.K), d.gated,
        static_cast<T*>(c.out), err);
    return cudaGetLastError();
  };
  return TM_BY_DTYPE(c.out_dtype, go);
}

tm_status mx_check(const tm_mxfp4* h, const MxCall& c, size_t ws_bytes) {
  const tm_mxfp4_desc& d = h->desc;
  if (!dtype_ok(c.x_dtype)) return status_fail(TM_EINVAL, "x dtype=%d is not a tm_dtype", c.x_dtype);
  if (!dtype_ok(c.out_dtype)) return status_fail(TM_EINVAL, "out dtype=%d is not a tm_dtype", c.out_dtype);
  if (c.ld < d.K) return status_fail(TM_EINVAL, "ld=%lld is less than K=%d", (long long)c.ld, d.K);
  if (!c.x || !c.out) return status_fail(TM_EINVAL, "x and out must be non-NULL");
  if (((uintptr_t)c.x) % dtype_bytes(c.x_dtype)) return status_fail(TM_EINVAL, "x must be aligned to its elements");
  if (((uintptr_t)c.out) % dtype_bytes(c.out_dtype))
    return status_fail(TM_EINVAL, "out must be aligned to its elements");
  if (c.rows > d.max_rows) return status_fail(TM_EINVAL, "%d rows exceed the prepared max_rows=%d", c.rows, d.max_rows);
  if (!c.ws) return status_fail(TM_EWORKSPACE, "workspace is NULL");
  if (((uintptr_t)c.ws) % kMxAlign) return status_fail(TM_EWORKSPACE, "workspace must be %zu-byte aligned", kMxAlign);
  const size_t need = mx_layout(d, c.rows).total;
  if (ws_bytes < need)
    return status_fail(TM_EWORKSPACE, "workspace has %zu bytes, %zu needed for %d rows", ws_bytes, need, c.rows);
  return TM_OK;
}

}  // namespace

}  // namespace tmoe

using namespace tmoe;

extern "C" {

tm_status trellis_moe_mxfp4_prepare(const tm_mxfp4_desc* desc, tm_mxfp4** out, size_t* workspace_bytes) {
  set_last_error("");
  if (out) *out = nullptr;
  if (!desc || !out) return status_fail(TM_EINVAL, "desc and out must be non-NULL");
  const tm_mxfp4_desc& d = *desc;
  if (d.E < 1 || d.E > kMaxExperts) return status_fail(TM_EUNSUPPORTED, "E=%d outside 1..%d", d.E, kMaxExperts);
  if (d.N < 1 || d.N > (1 << 20)) return status_fail(TM_EUNSUPPORTED, "N=%d outside 1..%d", d.N, 1 << 20);
  if (d.K < 1 || d.K > (1 << 20)) return status_fail(TM_EUNSUPPORTED, "K=%d outside 1..%d", d.K, 1 << 20);
  if (d.gated != 0 && d.gated != 1) return status_fail(TM_EINVAL, "gated=%d must be 0 or 1", d.gated);
  if (d.max_rows < 1 || d.max_rows > (1 << 24))
    return status_fail(TM_EINVAL, "max_rows=%d outside 1..%d", d.max_rows, 1 << 24);
  if (!d.codes || ((uintptr_t)d.codes) % 16) return status_fail(TM_EINVAL, "codes must be non-NULL and 16-byte aligned");
  if (!d.scales) return status_fail(TM_EINVAL, "scales is NULL");
  tm_mxfp4* h = new (std::nothrow) tm_mxfp4();
  if (!h) return status_fail(TM_EINVAL, "out of host memory");
  h->desc = d;
  *out = h;
  if (workspace_bytes) *workspace_bytes = mx_layout(d, d.max_rows).total;
  return TM_OK;
}

size_t trellis_moe_mxfp4_workspace_size(const tm_mxfp4* h, int32_t rows) {
  if (!h || rows < 0) return 0;
  return mx_layout(h->desc, rows).total;
}

tm_status trellis_moe_mxfp4_forward(tm_mxfp4* h, const void* x, int32_t x_dtype, int64_t ld, int32_t T, void* out,
                                    int32_t out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  set_last_error("");
  if (!h) return status_fail(TM_EINVAL, "handle is NULL");
  if (h->desc.E != 1) return status_fail(TM_EINVAL, "the handle has %d experts: use the expert form", h->desc.E);
  if (T < 0) return status_fail(TM_EINVAL, "T=%d < 0", T);
  if (T == 0) return TM_OK;
  const MxCall c{x, x_dtype, ld, nullptr, T, T, 1, out, out_dtype, workspace};
  const tm_status s = mx_check(h, c, workspace_bytes);
  if (s != TM_OK) return s;
  const cudaError_t e = mx_run(h->desc, c, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "MXFP4 product");
}

tm_status trellis_moe_mxfp4_forward_experts(tm_mxfp4* h, const void* x, int32_t x_dtype, int64_t ld,
                                            int32_t per_route, const int32_t* ids, int32_t T, int32_t topk, void* out,
                                            int32_t out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  set_last_error("");
  if (!h) return status_fail(TM_EINVAL, "handle is NULL");
  if (per_route != 0 && per_route != 1) return status_fail(TM_EINVAL, "per_route=%d must be 0 or 1", per_route);
  if (T < 0) return status_fail(TM_EINVAL, "T=%d < 0", T);
  if (topk < 1 || topk > 32) return status_fail(TM_EINVAL, "topk=%d outside 1..32", topk);
  if (T == 0) return TM_OK;
  if ((long)T * topk > h->desc.max_rows)
    return status_fail(TM_EINVAL, "T*topk=%ld exceeds the prepared max_rows=%d", (long)T * topk, h->desc.max_rows);
  if (!ids) return status_fail(TM_EINVAL, "ids is NULL");
  const MxCall c{x, x_dtype, ld, ids, T * topk, per_route ? T * topk : T, per_route ? 1 : topk, out, out_dtype, workspace};
  const tm_status s = mx_check(h, c, workspace_bytes);
  if (s != TM_OK) return s;
  const cudaError_t e = mx_run(h->desc, c, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "MXFP4 expert products");
}

tm_status trellis_moe_mxfp4_poll_error(tm_mxfp4* h, void* workspace, uint32_t* flags, void* stream) {
  set_last_error("");
  if (!h || !workspace || !flags) return status_fail(TM_EINVAL, "NULL argument");
  cudaStream_t st = (cudaStream_t)stream;
  uint32_t v = 0;
  cudaError_t e;
  if ((e = cudaMemcpyAsync(&v, workspace, 4, cudaMemcpyDeviceToHost, st)) != cudaSuccess) return status_cuda(e, "read error word");
  if ((e = cudaStreamSynchronize(st)) != cudaSuccess) return status_cuda(e, "synchronize");
  if ((e = cudaMemsetAsync(workspace, 0, 4, st)) != cudaSuccess) return status_cuda(e, "clear error word");
  *flags = v;
  if (v != 0)
    return status_fail(TM_EDEVICE, "device error flags 0x%x (bit 0: expert id out of range; bit 1: a pipeline wait gave up)", v);
  return TM_OK;
}

void trellis_moe_mxfp4_destroy(tm_mxfp4* h) { delete h; }

}  // extern "C"
