// Products with MXFP4 weights (sm_103a): y = deq(q(x)) deq(W)^T for a dense
// matrix or for each route's expert, with the rows of x quantised to MXFP4 in
// the call. Entry points, workspace and the order of the kernels; the products
// themselves are in mxfp4_tc.cu.
#include <algorithm>
#include <new>

#include "mxfp4.h"
#include "status.h"

struct tm_mxfp4 {
  tm_mxfp4_desc desc;
  uint8_t* d_scales;  // the weights' scales as the tensor cores read them
  int sms;
  uint64_t wait_ns;   // trellis_moe_mxfp4_set_wait_test
  int stall;          // 0, or which wait of the kernels never ends by itself (same)
  CUtensorMap wmap;
};

namespace tmoe {

namespace {

constexpr size_t kMxAlign = 256;
size_t mx_align(size_t v) { return (v + kMxAlign - 1) / kMxAlign * kMxAlign; }

constexpr int kMxRowsMax = 240, kMxRowsMaxGated = 112;  // rows of a block (mxfp4_tc.cu)

struct MxCall {
  const void* x;
  int x_dtype;
  int64_t ld;
  const int32_t* ids;
  int rows;    // rows of y
  int x_rows;
  int topk;    // rows of y that read one row of x
  void* out;
  int out_dtype;
  void* ws;
};

// Rows of a block. Dense: as few blocks as the limit allows, evenly filled.
// By expert: the limit, or less where experts average fewer routes.
int mx_block_rows(const tm_mxfp4_desc& d, bool dense, long rows) {
  const int most = d.gated ? kMxRowsMaxGated : kMxRowsMax;
  long want = rows;
  if (dense) {
    const long blocks = (rows + most - 1) / most;
    want = (rows + blocks - 1) / blocks;
  } else {
    want = std::max<long>(16, 2 * rows / d.E);
  }
  return (int)std::min<long>(most, (want + 15) / 16 * 16);
}

long mx_max_blocks(const tm_mxfp4_desc& d, long rows, int bn) { return rows / bn + std::min<long>(d.E, rows) + 1; }

// Error word | route map | codes of x in block order | their scales. Sized for
// the largest block and for the most blocks, so that a workspace for more rows
// fits fewer.
struct MxLayout {
  size_t block_info, nblocks, route_of_slot, slot_of_route, codes, scales, total;
};

MxLayout mx_layout(const tm_mxfp4_desc& d, long rows) {
  MxLayout L;
  const long ex = std::min<long>(d.E, rows) + 1;
  const size_t slots = (size_t)(rows + ex * kMxRowsMax), blocks = (size_t)(rows / 16 + ex);
  const size_t B = mx_blocks(d.K), S = mx_stages(d.K);
  size_t o = kMxAlign;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += mx_align(bytes);
    return at;
  };
  const size_t R = (size_t)rows;
  L.block_info = take(blocks * 8);
  L.nblocks = take(4);
  L.route_of_slot = take(slots * 4);
  L.slot_of_route = take(R * 4);
  L.codes = take(slots * B * 16);
  L.scales = take(blocks * S * 1024 + slots / 128 * S * 1024);
  L.total = o;
  return L;
}

// Whether a call runs in the few-rows kernel (one launch, weights read once for
// each chunk of 16 rows, rows quantised in every CTA) rather than in the block
// kernel (quantisation and, by expert, a route map before it). us a call, few
// rows / blocks, bf16:
//   dense 4096 x 4096   T = 1: 6.8 / 7.8   4: 7.3 / 7.8   8: 9.4 / 7.8   16: 12.4 / 7.8
//   dense 1024 x 1024   T = 1: 3.8 / 5.2   4: 4.2 / 5.2   8: 5.3 / 5.2   16: 6.8 / 5.2
//   dense 5120 x 1536   T = 1: 5.2 / 5.8   4: 5.8 / 5.8   8: 8.2 / 5.8
//   128 experts, gated 1024 -> 512    64 routes: 7.1 / 10.9   128: 10.9 / 12.4   192: 13.9 / 12.4   256: 17.0 / 12.4
//   128 experts, 512 -> 1024          64 routes: 7.3 / 9.3    128: 10.3-11.2 / 10.8   192: 16.6 / 11.8
//   256 experts, gated 2048 -> 256    64 routes: 8.2 / 10.8   128: 9.3 / 13.4    256: 17.5 / 16.9
//   64 experts, gated 2560 -> 320     32 routes: 8.7 / 10.8   64: 13.4 / 11.4    96: 11.7 / 11.3
//   32 experts, 512 -> 2048           32 routes: 7.2 / 8.7    64: 9.2 / 8.8
//   16 experts, 4096 -> 768           16 routes: 8.2 / 10.3   32: 15.5 / 10.3
//   8 experts, gated 1024 -> 1024     16 routes: 5.7-7.3 / 8.8   32: 7.2-10.3 / 8.8
//   160 experts, 1536 -> 5120         16 routes: 12.3-14.0 / 15.4   32: 26.1 / 24.2-25.5    64: 42.6-47.8 / 40.2
// (Of these the rule errs by most, 18%, at 64 routes of 64 experts.) Hence, dense, up to 8 pieces (rows times stages) for a CTA to quantise, where
// the times are equal and the second launch's cost to the host is saved; by
// expert few rows each on average, and no more CTAs than a few waves.
bool mx_few_rows(const tm_mxfp4* h, const MxCall& c) {
  const tm_mxfp4_desc& d = h->desc;
  const long tiles = (d.N + 127) / 128;
  if (!c.ids) {
    const int stages = mx_stages(d.K), split = 1 << mx_dec_split(tiles, stages, h->sms);
    return c.rows <= 8 && c.rows * ((stages + split - 1) / split) <= 8;
  }
  return c.rows <= d.E + 8 && c.rows * tiles <= 8L * h->sms;
}

cudaError_t mx_run(tm_mxfp4* h, const MxCall& c, cudaStream_t st) {
  const tm_mxfp4_desc& d = h->desc;
  if (mx_few_rows(h, c)) {
    MxDecArgs a{};
    a.E = d.E;
    a.N = d.N;
    a.K = d.K;
    a.gated = d.gated;
    a.rows = c.rows;
    a.sms = h->sms;
    a.x = c.x;
    a.x_dtype = c.x_dtype;
    a.ld = c.ld;
    const int es = dtype_bytes(c.x_dtype);
    a.vec = ((uintptr_t)c.x) % 16 == 0 && (c.ld * es) % 16 == 0 && d.K % 8 == 0;  // (as eights())
    a.ids = c.ids;
    a.topk = c.topk;
    a.wscale = h->d_scales;
    a.out = c.out;
    a.out_dtype = c.out_dtype;
    a.err = static_cast<uint32_t*>(c.ws);
    a.wait_ns = h->wait_ns;
    a.stall_issuer = h->stall == 1;
    a.stall_epilogue = h->stall == 2;
    a.wmap = h->wmap;
    const int chunks = c.ids ? c.rows : 1;
    return launch_mx_dec(a, chunks, st);
  }
  const MxLayout L = mx_layout(d, c.rows);
  uint8_t* base = static_cast<uint8_t*>(c.ws);
  uint32_t* err = reinterpret_cast<uint32_t*>(base);
  auto i32 = [&](size_t off) { return reinterpret_cast<int32_t*>(base + off); };
  cudaError_t e;
  MxTcArgs a{};
  a.E = d.E;
  a.N = d.N;
  a.K = d.K;
  a.gated = d.gated;
  a.rows = c.rows;
  a.bn = mx_block_rows(d, c.ids == nullptr, c.rows);
  a.nrb = (a.bn + 127) / 128;
  a.wscale = h->d_scales;
  a.xscale = base + L.scales;
  a.out = c.out;
  a.err = err;
  a.sms = h->sms;
  a.wait_ns = h->wait_ns;
  a.stall_issuer = h->stall == 1;
  a.stall_epilogue = h->stall == 2;
  a.wmap = h->wmap;
  a.max_blocks = (c.rows + a.bn - 1) / a.bn;
  if (c.ids) {
    a.max_blocks = (int)mx_max_blocks(d, c.rows, a.bn);
    int2* info = reinterpret_cast<int2*>(base + L.block_info);
    a.block_info = info;
    a.nblocks = i32(L.nblocks);
    a.route_of_slot = i32(L.route_of_slot);
    const MxMapArgs rm{c.ids, c.rows, d.E, a.bn, info, i32(L.nblocks), i32(L.route_of_slot), i32(L.slot_of_route), err};
    if ((e = launch_mx_map(rm, st)) != cudaSuccess) return e;
  }
  MxQuantArgs q{c.x, c.ld, c.x_rows, d.K, c.topk, c.ids ? i32(L.slot_of_route) : nullptr, a.bn, a.nrb, base + L.codes,
                base + L.scales, c.out, d.N * dtype_bytes(c.out_dtype), err};
  if ((e = launch_mx_rows_quantize(q, c.x_dtype, st)) != cudaSuccess) return e;
  return launch_mx_tc(a, base + L.codes, (long)a.max_blocks * a.bn, c.out_dtype, st);
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
  if ((long)c.x_rows * mx_stages(d.K) > (1L << 30))
    return status_fail(TM_EUNSUPPORTED, "%d rows of K=%d are too large", c.x_rows, d.K);
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
  h->d_scales = nullptr;
  h->wait_ns = 0;
  h->stall = 0;
  const int halves = d.gated ? 2 : 1;
  cudaError_t e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
      (e = cudaMalloc(&h->d_scales, mx_weight_scale_bytes(d.E, halves, d.N, d.K))) != cudaSuccess ||
      (e = launch_mx_weight_scales(d.scales, d.E, halves, d.N, d.K, h->d_scales, nullptr)) != cudaSuccess ||
      (e = mx_weight_map(&h->wmap, d.codes, (long)d.E * halves * d.N, d.K)) != cudaSuccess ||
      (e = cudaStreamSynchronize(nullptr)) != cudaSuccess) {
    cudaFree(h->d_scales);
    delete h;
    return status_cuda(e, "lay out the scales");
  }
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
  const cudaError_t e = mx_run(h, c, (cudaStream_t)stream);
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
  const MxCall c{x, x_dtype, ld, ids, T * topk, per_route ? T * topk : T, per_route ? 1 : topk,
                 out, out_dtype, workspace};
  const tm_status s = mx_check(h, c, workspace_bytes);
  if (s != TM_OK) return s;
  const cudaError_t e = mx_run(h, c, (cudaStream_t)stream);
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

tm_status trellis_moe_mxfp4_set_wait_test(tm_mxfp4* h, uint64_t wait_limit_ns, int32_t stall) {
  set_last_error("");
  if (!h) return status_fail(TM_EINVAL, "handle is NULL");
  if (stall < 0 || stall > 2) return status_fail(TM_EINVAL, "stall=%d must be 0, 1 or 2", stall);
  h->wait_ns = wait_limit_ns;
  h->stall = stall;
  return TM_OK;
}

void trellis_moe_mxfp4_destroy(tm_mxfp4* h) {
  if (!h) return;
  cudaFree(h->d_scales);
  delete h;
}

}  // extern "C"
