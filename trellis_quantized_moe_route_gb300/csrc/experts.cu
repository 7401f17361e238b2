// Products by expert with 16-bit weights (sm_103a): entry points, the plan, the
// sum over a token's routes, and the kernel that takes any sizes and strides.
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

// ------------------------------------------------------- any sizes and strides
// C[i, j] = sum_k A(i, k) B(j, k) in 64 x 64 tiles by mma.sync, 32 of k at a
// time, operands read element by element and laid out k-major in shared memory.
// For rows that do not begin on 16 bytes (an odd K or N without padding, a column
// range at an odd place), which TMA cannot read. 25 to 30 TFLOP/s, bound by
// its loads of two bytes a lane.
//   forward  i: the expert's routes   j: n          k: k
//   grad_x   i: the expert's routes   j: k          k: n
//   grad_w   i: n                     j: k          k: the expert's routes
constexpr int kGenTile = 64, kGenStep = 32, kGenPad = 8, kGenThreads = 128;

template <typename T>
__device__ __forceinline__ void gen_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void gen_mma<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void gen_mma<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T, typename O, int MODE>
__global__ void __launch_bounds__(kGenThreads) k_ex_general(const ExArgs a) {
  __shared__ __align__(16) T sa[kGenTile][kGenStep + kGenPad];
  __shared__ __align__(16) T sb[kGenTile][kGenStep + kGenPad];
  __shared__ int s_off[kExMaxExperts + 2], s_first[kExMaxExperts + 2];
  __shared__ int s_row[kGenTile], s_src[kGenTile];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = a.T * a.topk, E = a.E;
  for (int e = tid; e <= E; e += kGenThreads) s_off[e] = a.offsets[e];
  if (tid == 0) s_off[E + 1] = R;
  __syncthreads();
  int expert, i0, I, J, depth;
  if (MODE == kExGradW) {
    expert = blockIdx.z;
    i0 = blockIdx.x * kGenTile;
    I = a.N, J = a.K, depth = s_off[expert + 1] - s_off[expert];
  } else {
    if (tid == 0) {
      int run = 0;
      for (int e = 0; e <= E; ++e) {
        s_first[e] = run;
        run += (s_off[e + 1] - s_off[e] + kGenTile - 1) / kGenTile;
      }
      s_first[E + 1] = run;
    }
    __syncthreads();
    const int b = blockIdx.x;
    if (b >= s_first[E + 1]) return;
    expert = 0;
    while (s_first[expert + 1] <= b) ++expert;
    i0 = (b - s_first[expert]) * kGenTile;
    I = s_off[expert + 1] - s_off[expert];
    J = MODE == kExForward ? a.N : a.K;
    depth = expert == E ? 0 : (MODE == kExForward ? a.K : a.N);  // (routes of no expert: zeros)
  }
  const int j0 = blockIdx.y * kGenTile, base = s_off[expert];
  if (MODE != kExGradW) {
    if (tid < kGenTile) s_row[tid] = i0 + tid < I ? a.order[base + i0 + tid] : -1;
    __syncthreads();
  }
  const T* x = static_cast<const T*>(a.x);
  const T* g = static_cast<const T*>(a.g);
  const T* w = static_cast<const T*>(a.w) + (size_t)(expert < E ? expert : 0) * a.lde;
  const T zero = from_f32<T>(0.0f);
  float acc[4][4][4] = {};  // [row pair of 16][column 8] of the warp's 32 x 32... (two row tiles, four column tiles)
  const int wi = (warp >> 1) * 32, wj = (warp & 1) * 32;
  for (int k0 = 0; k0 < depth; k0 += kGenStep) {
    __syncthreads();
    if (MODE == kExGradW && tid < kGenStep) {
      const int r = k0 + tid < depth ? a.order[base + k0 + tid] : -1;
      s_row[tid] = r;
      s_src[tid] = r < 0 || a.per_route ? r : r / a.topk;
    }
    if (MODE == kExGradW) __syncthreads();
    for (int q = tid; q < kGenTile * kGenStep; q += kGenThreads) {
      if (MODE == kExGradW) {  // neighbouring threads along the rows' columns
        const int i = q % kGenTile, k = q / kGenTile;
        const bool in = s_row[k] >= 0;
        sa[i][k] = in && i0 + i < I ? g[(size_t)s_row[k] * a.ldg + i0 + i] : zero;
        sb[i][k] = in && j0 + i < J ? x[(size_t)s_src[k] * a.ldx + j0 + i] : zero;
      } else {
        const int i = q / kGenStep, k = q % kGenStep;
        const int r = s_row[i];
        const bool in = r >= 0 && k0 + k < depth;
        if (MODE == kExForward)
          sa[i][k] = in ? x[(size_t)(a.per_route ? r : r / a.topk) * a.ldx + k0 + k] : zero;
        else
          sa[i][k] = in ? g[(size_t)r * a.ldg + k0 + k] : zero;
        if (MODE == kExForward) {
          sb[i][k] = j0 + i < J && k0 + k < depth ? w[(size_t)(j0 + i) * a.ldw + k0 + k] : zero;
        } else {
          const int j = q % kGenTile, n = q / kGenTile;
          sb[j][n] = j0 + j < J && k0 + n < depth ? w[(size_t)(k0 + n) * a.ldw + j0 + j] : zero;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kGenStep; kk += 16) {
      const int r = lane >> 2, c = kk + (lane & 3) * 2;
      uint32_t fa[2][4], fb[4][2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int i = wi + m * 16 + r;
        fa[m][0] = *reinterpret_cast<const uint32_t*>(&sa[i][c]);
        fa[m][1] = *reinterpret_cast<const uint32_t*>(&sa[i + 8][c]);
        fa[m][2] = *reinterpret_cast<const uint32_t*>(&sa[i][c + 8]);
        fa[m][3] = *reinterpret_cast<const uint32_t*>(&sa[i + 8][c + 8]);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        fb[n][0] = *reinterpret_cast<const uint32_t*>(&sb[wj + n * 8 + r][c]);
        fb[n][1] = *reinterpret_cast<const uint32_t*>(&sb[wj + n * 8 + r][c + 8]);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) gen_mma<T>(acc[m][n], fa[m], fb[n][0], fb[n][1]);
    }
  }
  O* out = static_cast<O*>(a.out);
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int i = wi + m * 16 + (lane >> 2) + (v >> 1) * 8, j = j0 + wj + n * 8 + (lane & 3) * 2 + (v & 1);
        if (i0 + i >= I || j >= J) continue;
        const size_t row = MODE == kExGradW ? (size_t)expert * a.N + i0 + i : (size_t)s_row[i];
        out[row * J + j] = from_f32<O>(acc[m][n][v]);
      }
}

template <typename T, typename O>
cudaError_t gen_launch(const ExArgs& a, cudaStream_t st) {
  const long R = (long)a.T * a.topk;
  const unsigned blocks = (unsigned)(R / kGenTile + std::min<long>(R, a.E + 1));  // (at least as many as there are)
  auto tiles = [](int n) { return (unsigned)((n + kGenTile - 1) / kGenTile); };
  if (a.mode == kExForward)
    k_ex_general<T, O, kExForward><<<dim3(blocks, tiles(a.N)), kGenThreads, 0, st>>>(a);
  else if (a.mode == kExGradX)
    k_ex_general<T, O, kExGradX><<<dim3(blocks, tiles(a.K)), kGenThreads, 0, st>>>(a);
  else
    k_ex_general<T, O, kExGradW><<<dim3(tiles(a.N), tiles(a.K), a.E), kGenThreads, 0, st>>>(a);
  return cudaGetLastError();
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
  return TM_BY_DTYPE_VEC(dtype, eights(rows, K, K, 4) && eights(out, K, K, dtype_bytes(dtype)), go);
}

cudaError_t launch_ex_general(const ExArgs& a, cudaStream_t st) {
  auto go = [&](auto elem) {
    using O = decltype(elem);
    return a.dtype == TM_BF16 ? gen_launch<__nv_bfloat16, O>(a, st) : gen_launch<__half, O>(a, st);
  };
  return TM_BY_DTYPE(a.out_dtype, go);
}

namespace {

cudaError_t ex_product(const ExArgs& a, cudaStream_t st) {
  if (!ex_tc_ok(a)) return launch_ex_general(a, st);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
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
  return TM_OK;
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
  const cudaError_t e = launch_ex_plan(ids, R, E, order, offsets, flags, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "expert plan");
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
  const tm_status s = ex_check(a);
  if (s != TM_OK || T == 0) return s;
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
  const tm_status s = ex_check(a);
  if (s != TM_OK || T == 0) return s;
  if (!per_route) {
    if (!grad_x || ((uintptr_t)grad_x) % 2) return status_fail(TM_EINVAL, "grad_x must be non-NULL and aligned to its elements");
    if (((uintptr_t)workspace) % 16) return status_fail(TM_EINVAL, "workspace must be 16-byte aligned");
    if (workspace_bytes < trellis_moe_experts_grad_x_workspace_size(T, topk, K, per_route))
      return status_fail(TM_EWORKSPACE, "workspace of %zu bytes is too small", workspace_bytes);
    if ((long)T * ((K + 7) / 8) >= 1L << 31) return status_fail(TM_EUNSUPPORTED, "T=%d rows of K=%d are too many", T, K);
  }
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
  const tm_status s = ex_check(a);
  if (s != TM_OK) return s;
  const cudaError_t e = ex_product(a, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "expert products' gradient of w");
}

}  // extern "C"
