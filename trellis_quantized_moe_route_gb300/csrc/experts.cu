// Products by expert with 16-bit weights (sm_103a): entry points, the plan, the
// sum over a token's routes, and copies of rows that TMA cannot read.
//   y_r = W_e x_s(r),   dx_s = sum of W_e^T dy_r over the routes r that read row s,
//   dW_e = sum of dy_r x_s(r)^T over the expert's routes, in order.
#include "experts.h"

#include <algorithm>

#include "elem.cuh"
#include "pdl.cuh"
#include "status.h"

namespace tmoe {

namespace {

constexpr int kExMaxExperts = 256;
constexpr int kExMaxSide = 1 << 20;  // N and K

// ------------------------------------------------------------------ the plan
// Routes sorted by expert, stably: their order is that of the sums in dW, which
// so do not depend on the run. A warp takes a stretch of the routes, 32 at a
// time: lanes of one expert find each other, the lowest adds their number to the
// warp's count. Counts are summed over the warps and the CTAs of the cluster, and
// the same walk gives every route its place. Ids outside 0..E-1 form a last
// group. Bound by latency: one CTA for up to kPlanAlone routes, a cluster beyond;
// what the first kPlanHeld steps found stays in registers. 8 routes: 4.6 us a call
// back to back, 64: 5.2, 5120: 6.7, 16384: 8.7, 32768: 10.6.
constexpr int kPlanThreads = 1024, kPlanFew = 512;  // of a CTA of the cluster, of the one CTA
constexpr int kPlanCtas = 8;
constexpr int kPlanHeld = 4;
constexpr int kPlanAlone = 2048;
constexpr int kPlanGroups = kExMaxExperts + 1;

__device__ __forceinline__ int plan_peer(const int* p, int rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];\n" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// The lanes with the same group, bit by bit. (match.any serves one warp of an SM
// at a time, some 70 cycles each: 32768 routes took 14.8 us.)
__device__ __forceinline__ uint32_t plan_same(int e, int bits) {
  uint32_t same = 0xFFFFFFFFu;
  for (int b = 0; b < bits; ++b) {
    const uint32_t v = __ballot_sync(0xFFFFFFFFu, e >> b & 1);
    same &= e >> b & 1 ? v : ~v;
  }
  return same;
}

template <int CTAS, int THREADS>
__global__ void __launch_bounds__(THREADS)
    k_ex_plan(const int32_t* __restrict__ ids, int R, int E, int32_t* __restrict__ order, int32_t* __restrict__ offsets,
              uint32_t* __restrict__ flags) {
  constexpr int kPlanWarps = THREADS / 32;
  __shared__ int s_cnt[kPlanWarps][kPlanGroups];  // counts, then places, by warp
  __shared__ int s_all[kPlanGroups];              // the CTA's counts
  __shared__ int s_scan[kPlanGroups], s_warp[kPlanWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = E + 1;
  uint32_t rank = 0;
  if (CTAS > 1) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  for (int i = tid; i < kPlanWarps * kPlanGroups; i += THREADS) (&s_cnt[0][0])[i] = 0;
  __syncthreads();
  grid_wait();
  grid_launch();
  const int per = (R + CTAS * kPlanWarps - 1) / (CTAS * kPlanWarps);  // routes of a warp
  const int lo = min((long)R, (long)per * (rank * kPlanWarps + warp)), hi = min(R, lo + per);
  const int bits = 32 - __clz(E + 1);  // (groups 0..E, and E + 1 for no route)
  auto group = [&](int r) {
    const int e = r < hi ? ids[r] : 0;
    return r < hi ? (e >= 0 && e < E ? e : E) : E + 1;
  };
  int held[kPlanHeld];
  uint32_t same[kPlanHeld];
#pragma unroll
  for (int u = 0; u < kPlanHeld; ++u) held[u] = group(lo + u * 32 + lane);
  auto count = [&](int e, uint32_t m) {
    if (e <= E && lane == __ffs(m) - 1) s_cnt[warp][e] += __popc(m);
    __syncwarp();
  };
#pragma unroll
  for (int u = 0; u < kPlanHeld; ++u)
    if (lo + u * 32 < hi) {
      same[u] = plan_same(held[u], bits);
      count(held[u], same[u]);
    }
  for (int r = lo + kPlanHeld * 32; r < hi; r += 32) {
    const int e = group(r + lane);
    count(e, plan_same(e, bits));
  }
  __syncthreads();
  int all = 0;
  if (tid < G) {
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
      const int c = s_cnt[w][tid];
      s_cnt[w][tid] = all;
      all += c;
    }
  }
  int before = 0, total = all;
  if (CTAS > 1) {
    if (tid < G) s_all[tid] = all;
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    if (tid < G) {
      int v[CTAS];
#pragma unroll
      for (int c = 0; c < CTAS; ++c) v[c] = plan_peer(&s_all[tid], c);
      total = 0;
#pragma unroll
      for (int c = 0; c < CTAS; ++c) {
        if (c < (int)rank) before += v[c];
        total += v[c];
      }
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");  // (done with the peers' counts)
  }
  // exclusive scan of the totals, one to a thread
  int incl = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  if (tid < G) {
    int first = incl - total;
    for (int w = 0; w < warp; ++w) first += s_warp[w];
    s_scan[tid] = first + before;
    if (rank == 0) {
      offsets[tid] = first;  // (offsets[E]: where the last group begins)
      if (tid == E) *flags = total ? 1u : 0u;
    }
  }
  __syncthreads();
  auto place = [&](int r, int e, uint32_t m) {
    if (e <= E) order[s_scan[e] + s_cnt[warp][e] + __popc(m & ((1u << lane) - 1))] = r;
    __syncwarp();
    count(e, m);
  };
#pragma unroll
  for (int u = 0; u < kPlanHeld; ++u)
    if (lo + u * 32 < hi) place(lo + u * 32 + lane, held[u], same[u]);
  for (int r = lo + kPlanHeld * 32; r < hi; r += 32) {
    const int e = group(r + lane);
    place(r + lane, e, plan_same(e, bits));
  }
  __syncwarp();
  if (CTAS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");  // no CTA leaves while another reads its counts
}

// ------------------------------------------------------------ aligned copies
// Rows that do not begin on 16 bytes (an odd N or K without padding, a column range
// at an odd place) cannot be read by TMA; copies of them can. Eight elements come
// as the one or two aligned words of 16 bytes that hold them, shifted into place.
// Bound by memory: some 5.7 TB/s read and written. Products with their copies,
// forward, dx, dW in us: 5120 routes of 64 experts, 2559 -> 641, 112, 138, 112 (aligned
// 42, 64, 50; by mma.sync in tiles of 128, with the shifting in its loads, 429, 316, 398);
// 8192 of 4 experts, 2049 -> 2047, 89, 123 to 131, 94 (592, 597, 562); 64 of 128 experts, 1025 ->
// 1023, 64 to 73, 67 to 77, 118 (138, 139, 315).
constexpr int kAlignThreads = 256, kAlignWords = 4;  // of a thread

struct ExAlignJob {
  const uint16_t* src;
  uintptr_t lo, hi;    // the memory that src's rows and what lies between them take
  int64_t ld, lde;     // elements between rows and between matrices
  FastDiv words;       // 16-byte words of a row of the copy
  uint32_t total;      // words of a matrix
  uint32_t ctas;       // that copy a matrix
  int cols;
  uint4* dst;
};

// CTAs in a list: each expert's w's, then x's, then g's. (As many for each expert as
// the largest tensor needs, 32768 rows and 160 experts, 2559 -> 641, were 1650000 CTAs, of which
// 42000 had work: 1.86 ms for the forward call, 0.37 so.)
struct ExAlignArgs {
  ExAlignJob w, x, g;  // E matrices, one and one; those that are not copied: no CTAs
  uint32_t w_ctas;     // of all experts
  FastDiv per_expert;
  const int32_t* offsets;
};

// n (at most eight) elements of 16 bits at p, then zeros.
__device__ __forceinline__ uint4 align_load(const uint16_t* p, int n, uintptr_t lo, uintptr_t hi) {
  const uintptr_t at = (uintptr_t)p, w0 = at & ~(uintptr_t)15;
  const int off = (int)(at & 15);
  const bool two = off + 2 * n > 16;
  if (w0 >= lo && w0 + (two ? 32 : 16) <= hi) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(w0));
    const uint4 y = two ? __ldg(reinterpret_cast<const uint4*>(w0) + 1) : make_uint4(0, 0, 0, 0);
    // the words from byte `off` on, by 8, 4 and 2 bytes
    const bool e = off & 8, f = off & 4;
    const uint32_t a0 = e ? x.z : x.x, a1 = e ? x.w : x.y, a2 = e ? y.x : x.z, a3 = e ? y.y : x.w, a4 = e ? y.z : y.x, a5 = e ? y.w : y.y;
    const uint32_t b0 = f ? a1 : a0, b1 = f ? a2 : a1, b2 = f ? a3 : a2, b3 = f ? a4 : a3, b4 = f ? a5 : a4;
    const int s = (off & 2) * 8;
    return make_uint4(__funnelshift_r(b0, b1, s), __funnelshift_r(b1, b2, s), __funnelshift_r(b2, b3, s), __funnelshift_r(b3, b4, s));
  }
  uint32_t w[4] = {};  // (the tensor's first and last words)
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i >> 1] |= (uint32_t)__ldg(p + i) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(kAlignThreads) k_ex_align(const __grid_constant__ ExAlignArgs a) {
  grid_wait();
  grid_launch();
  uint32_t b = blockIdx.x, e = 0;
  const bool w = b < a.w_ctas;
  if (w) {
    e = a.per_expert.div(b);
    b -= e * a.per_expert.d;
    if (a.offsets[e] == a.offsets[e + 1]) return;  // (nobody reads it)
  } else {
    b -= a.w_ctas;
  }
  const bool x = !w && b < a.x.ctas;
  if (!w && !x) b -= a.x.ctas;
  const ExAlignJob& j = w ? a.w : x ? a.x : a.g;
  const uint16_t* src = j.src + (size_t)e * j.lde;
  uint4* dst = j.dst + (size_t)e * j.total;
  const uint32_t n0 = b * (kAlignThreads * kAlignWords) + threadIdx.x;
  uint4 q[kAlignWords];
#pragma unroll
  for (int u = 0; u < kAlignWords; ++u) {
    const uint32_t n = n0 + u * kAlignThreads;
    if (n < j.total) {
      const uint32_t row = j.words.div(n), c = (n - row * j.words.d) * 8;
      q[u] = align_load(src + (size_t)row * j.ld + c, min(8, j.cols - (int)c), j.lo, j.hi);
    }
  }
#pragma unroll
  for (int u = 0; u < kAlignWords; ++u)
    if (n0 + u * kAlignThreads < j.total) dst[n0 + u * kAlignThreads] = q[u];
}

// A thread takes eight columns of a token. The routes' rows are in fp32, so that a
// token's sum is rounded once; bound by their bytes, which mostly come from L2.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_ex_sum(const float* __restrict__ rows, uint32_t total, FastDiv per, int topk, int K,
                                                T* __restrict__ out) {
  grid_wait();
  grid_launch();
  const uint32_t n = blockIdx.x * 256 + threadIdx.x;
  if (n >= total) return;
  const size_t t = per.div(n);
  const int c = (int)(n - (uint32_t)t * per.d) * 8, len = min(8, K - c);
  float acc[8] = {};
  const float* row = rows + t * topk * K + c;
  for (int j0 = 0; j0 < topk; j0 += 4) {
    Eight<float, VEC> e[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) e[u].load(row + (size_t)(j0 + u) * K, j0 + u < topk ? len : 0);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float v[8];
      e[u].to(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[i];
    }
  }
  Eight<T, VEC> o;
  o.from(acc);
  o.store(out + t * K + c, len);
}

}  // namespace

cudaError_t launch_ex_plan(const int32_t* ids, int R, int E, int32_t* order, int32_t* offsets, uint32_t* flags,
                           cudaStream_t st) {
  if (R <= kPlanAlone) return launch_after(k_ex_plan<1, kPlanFew>, dim3(1), kPlanFew, 0, st, ids, R, E, order, offsets, flags);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kPlanCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = kPlanCtas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_ex_plan<kPlanCtas, kPlanThreads>, ids, R, E, order, offsets, flags);
}

cudaError_t launch_ex_sum(const float* rows, int T, int topk, int K, void* out, int dtype, cudaStream_t st) {
  const int per = (K + 7) / 8;
  const long total = (long)T * per;  // (below 2^31 by the entry point's checks)
  auto go = [&](auto elem, auto vec) {
    using O = decltype(elem);
    return launch_after(k_ex_sum<O, decltype(vec)::value>, dim3((unsigned)((total + 255) / 256)), 256, 0, st, rows,
                        (uint32_t)total, FastDiv(per), topk, K, static_cast<O*>(out));
  };
  const bool vec = eights(rows, K, K, 4) && eights(out, K, K, 2);  // (dx is of 16 bits)
  auto with = [&](auto elem) { return vec ? go(elem, std::true_type()) : go(elem, std::false_type()); };
  return dtype == TM_BF16 ? with(__nv_bfloat16()) : with(__half());
}

namespace {

// trellis_moe_experts_set_wait_test, by thread (there is no handle that could hold it).
struct ExWaitTest {
  uint64_t wait_ns;
  int stall;
};
thread_local ExWaitTest ex_wait_test;

cudaError_t ex_product(ExArgs a, cudaStream_t st) {
  a.wait_ns = ex_wait_test.wait_ns, a.stall = ex_wait_test.stall;
  if (a.T == 0)  // (grad_w of no tokens)
    return cudaMemsetAsync(a.out, 0, (size_t)a.E * a.N * a.K * dtype_bytes(a.out_dtype), st);
  int sms = 0;
  const cudaError_t e = current_sms(sms);
  return e == cudaSuccess ? launch_ex_tc(a, sms, st) : e;
}

tm_status ex_check(const ExArgs& a) {
  if (a.dtype != TM_BF16 && a.dtype != TM_F16) return status_fail(TM_EINVAL, "dtype=%d is not TM_BF16 or TM_F16", a.dtype);
  if (!dtype_ok(a.out_dtype)) return status_fail(TM_EINVAL, "out_dtype=%d is not a tm_dtype", a.out_dtype);
  if (a.T < 0) return status_fail(TM_EINVAL, "T=%d < 0", a.T);
  if (a.topk < 1 || a.topk > 32) return status_fail(TM_EINVAL, "topk=%d outside 1..32", a.topk);
  if (a.E < 1 || a.E > kExMaxExperts) return status_fail(TM_EUNSUPPORTED, "E=%d outside 1..%d", a.E, kExMaxExperts);
  if (a.N < 1 || a.N > kExMaxSide) return status_fail(TM_EINVAL, "N=%d outside 1..%d", a.N, kExMaxSide);
  if (a.K < 1 || a.K > kExMaxSide) return status_fail(TM_EINVAL, "K=%d outside 1..%d", a.K, kExMaxSide);
  if ((long)a.T * a.topk > (1 << 22)) return status_fail(TM_EUNSUPPORTED, "T * topk = %ld routes: more than %d", (long)a.T * a.topk, 1 << 22);
  if (a.per_route != 0 && a.per_route != 1) return status_fail(TM_EINVAL, "per_route=%d must be 0 or 1", a.per_route);
  if (a.mode != kExGradX && a.ldx < a.K) return status_fail(TM_EINVAL, "ldx=%lld is less than K=%d", (long long)a.ldx, a.K);
  if (a.mode != kExForward && a.ldg < a.N) return status_fail(TM_EINVAL, "ldg=%lld is less than N=%d", (long long)a.ldg, a.N);
  if (a.mode != kExGradW && (a.ldw < a.K || a.lde < 0))
    return status_fail(TM_EINVAL, "ldw=%lld, lde=%lld: rows of w must not overlap", (long long)a.ldw, (long long)a.lde);
  if (a.T == 0 && a.mode != kExGradW) return TM_OK;
  const bool in = a.T == 0 || ((a.mode == kExGradX || a.x) && (a.mode == kExForward || a.g));
  if (!in || (a.mode != kExGradW && !a.w) || !a.out || (a.T > 0 && !a.order) || !a.offsets || !a.flags)
    return status_fail(TM_EINVAL, "arguments must be non-NULL");
  const void* p[] = {a.x, a.g, a.w};
  for (const void* q : p)
    if (((uintptr_t)q) % 2) return status_fail(TM_EINVAL, "x, w and grad_out must be aligned to their elements");
  if (((uintptr_t)a.out) % dtype_bytes(a.out_dtype)) return status_fail(TM_EINVAL, "the result must be aligned to its elements");
  auto rows_ok = [](const void* q, int64_t ld) { return ((uintptr_t)q) % 16 == 0 && ld % 8 == 0 && ld < (1LL << 38); };
  if (a.T > 0 && ((a.mode != kExGradX && !rows_ok(a.x, a.ldx)) || (a.mode != kExForward && !rows_ok(a.g, a.ldg)) ||
                  (a.mode != kExGradW && (!rows_ok(a.w, a.ldw) || (a.E > 1 && (!rows_ok(a.w, a.lde) || a.lde == 0))))))
    return status_fail(TM_EINVAL, "rows of x, w and grad_out must begin on 16 bytes (trellis_moe_experts_align copies them so)");
  return TM_OK;
}

// Whether [lo, hi) touches any of E matrices, lde elements of 16 bits apart, of
// `rows` rows of `cols` elements, ld apart. (It may lie between the rows.)
bool ex_touch(uintptr_t lo, uintptr_t hi, const void* src, int64_t ld, int64_t lde, int E, int64_t rows, int64_t cols) {
  const uintptr_t p = (uintptr_t)src, row = (uintptr_t)cols * 2, step = (uintptr_t)ld * 2;
  if (!src || lo >= hi || p >= hi || p + ((uintptr_t)(E - 1) * lde + (uintptr_t)(rows - 1) * ld) * 2 + row <= lo) return false;
  for (int e = 0; e < E; ++e) {
    const uintptr_t q = p + (uintptr_t)e * lde * 2;
    const uintptr_t r = lo < q + row ? 0 : (lo - q - row) / step + 1;  // the first row that ends behind lo
    if (r < (uintptr_t)rows && q + r * step < hi) return true;
  }
  return false;
}

bool ex_meet(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  return a_bytes && b_bytes && (uintptr_t)a < (uintptr_t)b + b_bytes && (uintptr_t)b < (uintptr_t)a + a_bytes;
}

// A product's CTAs store rows while others still read theirs.
tm_status ex_check_apart(const ExArgs& a) {
  const int64_t R = (int64_t)a.T * a.topk, xrows = a.per_route ? R : a.T;
  const size_t rows = a.mode == kExGradW ? (size_t)a.E * a.N : (size_t)R, cols = a.mode == kExForward ? a.N : a.K;
  const size_t bytes = rows * cols * dtype_bytes(a.out_dtype);
  const uintptr_t lo = (uintptr_t)a.out, hi = lo + bytes;
  const bool meets = (a.mode != kExGradX && ex_touch(lo, hi, a.x, a.ldx, 0, 1, xrows, a.K)) ||
                     (a.mode != kExForward && ex_touch(lo, hi, a.g, a.ldg, 0, 1, R, a.N)) ||
                     (a.mode != kExGradW && ex_touch(lo, hi, a.w, a.ldw, a.lde, a.E, a.N, a.K)) ||
                     ex_meet(a.out, bytes, a.order, (size_t)R * 4) || ex_meet(a.out, bytes, a.offsets, (size_t)(a.E + 1) * 4) ||
                     ex_meet(a.out, bytes, a.flags, 4);
  return meets ? status_fail(TM_EINVAL, "the result (or workspace) must not overlap x, w, grad_out or the plan") : TM_OK;
}

// One tensor of an aligned copy: E matrices of `rows` rows; false if it is too large.
bool ex_align_job(ExAlignJob& j, const void* src, int64_t ld, int64_t lde, int E, int rows, int cols, void* dst) {
  const int words = (cols + 7) / 8;
  const long total = (long)rows * words;
  j.src = static_cast<const uint16_t*>(src), j.ld = ld, j.lde = lde, j.cols = cols, j.dst = static_cast<uint4*>(dst);
  j.words = FastDiv((uint32_t)words), j.total = (uint32_t)total;
  j.ctas = (uint32_t)((total + kAlignThreads * kAlignWords - 1) / (kAlignThreads * kAlignWords));  // (below 2^21)
  j.lo = (uintptr_t)src;
  j.hi = (uintptr_t)(j.src + (int64_t)(E - 1) * lde + (int64_t)(rows - 1) * ld + cols);
  return total < 1L << 31;
}

}  // namespace

}  // namespace tmoe

using namespace tmoe;

extern "C" {

tm_status trellis_moe_expert_plan(const int32_t* ids, int32_t R, int32_t E, int32_t* order, int32_t* offsets,
                                  uint32_t* flags, void* stream) {
  set_last_error("");
  if (R < 0 || R > (1 << 22)) return status_fail(TM_EUNSUPPORTED, "%d routes: outside 0..%d", R, 1 << 22);
  if (E < 1 || E > kExMaxExperts) return status_fail(TM_EUNSUPPORTED, "E=%d outside 1..%d", E, kExMaxExperts);
  if ((R > 0 && (!ids || !order)) || !offsets || !flags) return status_fail(TM_EINVAL, "ids, order, offsets and flags must be non-NULL");
  const size_t rb = (size_t)R * 4, ob = (size_t)(E + 1) * 4;
  if (ex_meet(ids, rb, order, rb) || ex_meet(ids, rb, offsets, ob) || ex_meet(ids, rb, flags, 4) || ex_meet(order, rb, offsets, ob) ||
      ex_meet(order, rb, flags, 4) || ex_meet(offsets, ob, flags, 4))
    return status_fail(TM_EINVAL, "ids, order, offsets and flags must not overlap");
  const cudaError_t e = launch_ex_plan(ids, R, E, order, offsets, flags, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "expert plan");
}

tm_status trellis_moe_experts_align(const void* x, int64_t ldx, int32_t x_rows, const void* grad_out, int64_t ldg,
                                    int32_t g_rows, const void* w, int64_t ldw, int64_t lde, const int32_t* offsets, int32_t E,
                                    int32_t N, int32_t K, void* x_to, void* g_to, void* w_to, void* stream) {
  set_last_error("");
  if (E < 1 || E > kExMaxExperts) return status_fail(TM_EUNSUPPORTED, "E=%d outside 1..%d", E, kExMaxExperts);
  if (N < 1 || N > kExMaxSide) return status_fail(TM_EINVAL, "N=%d outside 1..%d", N, kExMaxSide);
  if (K < 1 || K > kExMaxSide) return status_fail(TM_EINVAL, "K=%d outside 1..%d", K, kExMaxSide);
  if ((x_to && x_rows < 1) || (g_to && g_rows < 1)) return status_fail(TM_EINVAL, "x_rows=%d, g_rows=%d: less than 1", x_rows, g_rows);
  if (x_to && ldx < K) return status_fail(TM_EINVAL, "ldx=%lld is less than K=%d", (long long)ldx, K);
  if (g_to && ldg < N) return status_fail(TM_EINVAL, "ldg=%lld is less than N=%d", (long long)ldg, N);
  if (w_to && (ldw < K || lde < 0))
    return status_fail(TM_EINVAL, "ldw=%lld, lde=%lld: rows of w must not overlap", (long long)ldw, (long long)lde);
  if ((x_to && !x) || (g_to && !grad_out) || (w_to && (!w || !offsets))) return status_fail(TM_EINVAL, "arguments must be non-NULL");
  for (const void* q : {x_to ? x : nullptr, g_to ? grad_out : nullptr, w_to ? w : nullptr})
    if (((uintptr_t)q) % 2) return status_fail(TM_EINVAL, "x, w and grad_out must be aligned to their elements");
  for (const void* q : {x_to, g_to, w_to})
    if (((uintptr_t)q) % 16) return status_fail(TM_EINVAL, "the copies must be 16-byte aligned");
  ExAlignArgs a{ExAlignJob{.words = FastDiv(1)}, ExAlignJob{.words = FastDiv(1)}, ExAlignJob{.words = FastDiv(1)}, 0, FastDiv(1), offsets};
  const bool ok = (!x_to || ex_align_job(a.x, x, ldx, 0, 1, x_rows, K, x_to)) &&
                  (!g_to || ex_align_job(a.g, grad_out, ldg, 0, 1, g_rows, N, g_to)) &&
                  (!w_to || ex_align_job(a.w, w, ldw, lde, E, N, K, w_to));
  const struct {
    const void* p;
    size_t bytes;
  } to[3] = {{x_to, (size_t)a.x.total * 16}, {g_to, (size_t)a.g.total * 16}, {w_to, (size_t)a.w.total * 16 * E}};
  bool meets = false;
  for (int i = 0; ok && i < 3; ++i) {
    if (!to[i].p) continue;
    const uintptr_t lo = (uintptr_t)to[i].p, hi = lo + to[i].bytes;
    meets = meets || (x_to && ex_touch(lo, hi, x, ldx, 0, 1, x_rows, K)) || (g_to && ex_touch(lo, hi, grad_out, ldg, 0, 1, g_rows, N)) ||
            (w_to && (ex_touch(lo, hi, w, ldw, lde, E, N, K) || ex_meet(to[i].p, to[i].bytes, offsets, (size_t)(E + 1) * 4)));
    for (int j = 0; j < i; ++j) meets = meets || (to[j].p && ex_meet(to[i].p, to[i].bytes, to[j].p, to[j].bytes));
  }
  if (meets) return status_fail(TM_EINVAL, "the copies must not overlap what is copied, or one another");
  if (!ok) return status_fail(TM_EUNSUPPORTED, "a matrix of 2^34 elements or more cannot be copied");
  if (w_to) a.w_ctas = a.w.ctas * (uint32_t)E, a.per_expert = FastDiv(a.w.ctas);
  const uint32_t ctas = a.w_ctas + a.x.ctas + a.g.ctas;  // (below 2^30)
  if (ctas == 0) return TM_OK;
  const cudaError_t e = launch_after(k_ex_align, dim3(ctas), kAlignThreads, 0, (cudaStream_t)stream, a);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "aligned copies");
}

tm_status trellis_moe_experts_forward(const void* x, int32_t dtype, int64_t ldx, int32_t per_route, const void* w,
                                      int64_t ldw, int64_t lde, const int32_t* order, const int32_t* offsets, int32_t T,
                                      int32_t topk, int32_t E, int32_t N, int32_t K, void* out, int32_t out_dtype,
                                      uint32_t* flags, void* stream) {
  set_last_error("");
  ExArgs a{};
  a.mode = kExForward, a.dtype = dtype, a.out_dtype = out_dtype, a.T = T, a.topk = topk, a.E = E, a.N = N, a.K = K;
  a.per_route = per_route, a.x = x, a.ldx = ldx, a.w = w, a.ldw = ldw, a.lde = lde, a.order = order, a.offsets = offsets;
  a.out = out, a.flags = flags;
  tm_status s = ex_check(a);
  if (s != TM_OK || T == 0) return s;
  if ((s = ex_check_apart(a)) != TM_OK) return s;
  const cudaError_t e = ex_product(a, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "expert products");
}

size_t trellis_moe_experts_grad_x_workspace_size(int32_t T, int32_t topk, int32_t K, int32_t per_route) {
  return per_route || T <= 0 || topk <= 0 || K <= 0 ? 0 : (size_t)T * topk * K * 4;
}

tm_status trellis_moe_experts_grad_x(const void* grad_out, int32_t dtype, int64_t ldg, int32_t per_route, const void* w,
                                     int64_t ldw, int64_t lde, const int32_t* order, const int32_t* offsets, int32_t T,
                                     int32_t topk, int32_t E, int32_t N, int32_t K, void* grad_x, uint32_t* flags,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  set_last_error("");
  ExArgs a{};
  a.mode = kExGradX, a.dtype = dtype, a.out_dtype = per_route ? dtype : TM_F32, a.T = T, a.topk = topk, a.E = E, a.N = N, a.K = K;
  a.per_route = per_route, a.g = grad_out, a.ldg = ldg, a.w = w, a.ldw = ldw, a.lde = lde, a.order = order, a.offsets = offsets;
  a.out = per_route ? grad_x : workspace, a.flags = flags;
  tm_status s = ex_check(a);
  if (s != TM_OK || T == 0) return s;
  if (!per_route) {
    if (!grad_x || ((uintptr_t)grad_x) % 2) return status_fail(TM_EINVAL, "grad_x must be non-NULL and aligned to its elements");
    if (((uintptr_t)workspace) % 16) return status_fail(TM_EINVAL, "workspace must be 16-byte aligned");
    if (workspace_bytes < trellis_moe_experts_grad_x_workspace_size(T, topk, K, per_route))
      return status_fail(TM_EWORKSPACE, "workspace of %zu bytes is too small", workspace_bytes);
    if ((long)T * ((K + 7) / 8) >= 1L << 31) return status_fail(TM_EUNSUPPORTED, "T=%d rows of K=%d are too many", T, K);
    // (written when the products are done; the plan stays whole for the next one)
    const size_t gb = (size_t)T * K * 2, rb = (size_t)T * topk * 4;
    if (ex_meet(grad_x, gb, workspace, rb * K) || ex_meet(grad_x, gb, order, rb) || ex_meet(grad_x, gb, offsets, (size_t)(E + 1) * 4) ||
        ex_meet(grad_x, gb, flags, 4))
      return status_fail(TM_EINVAL, "grad_x must not overlap the workspace or the plan");
  }
  if ((s = ex_check_apart(a)) != TM_OK) return s;
  cudaError_t e = ex_product(a, (cudaStream_t)stream);
  if (e == cudaSuccess && !per_route)
    e = launch_ex_sum(static_cast<const float*>(workspace), T, topk, K, grad_x, dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "expert products' gradient of x");
}

tm_status trellis_moe_experts_grad_w(const void* x, int32_t dtype, int64_t ldx, int32_t per_route, const void* grad_out,
                                     int64_t ldg, const int32_t* order, const int32_t* offsets, int32_t T, int32_t topk,
                                     int32_t E, int32_t N, int32_t K, void* grad_w, int32_t grad_dtype, uint32_t* flags,
                                     void* stream) {
  set_last_error("");
  ExArgs a{};
  a.mode = kExGradW, a.dtype = dtype, a.out_dtype = grad_dtype, a.T = T, a.topk = topk, a.E = E, a.N = N, a.K = K;
  a.per_route = per_route, a.x = x, a.ldx = ldx, a.g = grad_out, a.ldg = ldg, a.order = order, a.offsets = offsets;
  a.out = grad_w, a.flags = flags;
  tm_status s = ex_check(a);
  if (s == TM_OK && T > 0) s = ex_check_apart(a);
  if (s != TM_OK) return s;
  const cudaError_t e = ex_product(a, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "expert products' gradient of w");
}

tm_status trellis_moe_experts_set_wait_test(uint64_t wait_limit_ns, int32_t stall) {
  set_last_error("");
  if (stall < 0 || stall > 5) return status_fail(TM_EINVAL, "stall=%d outside 0..5", stall);
  ex_wait_test = {wait_limit_ns, stall};
  return TM_OK;
}

}  // extern "C"
