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
// C[i, j] = sum_k A(i, k) B(j, k) in 128 x 128 tiles by mma.sync, 32 of k at a time.
//   forward  i: the expert's routes   j: n          k: k                     both stored along k
//   grad_x   i: the expert's routes   j: k          k: n                     B stored along j
//   grad_w   i: n                     j: k          k: the expert's routes   both stored along i, j
// For rows that do not begin on 16 bytes (an odd K or N without padding, a column
// range at an odd place), which TMA cannot read: eight elements come as the one or
// two aligned words of 16 bytes that hold them, shifted into place, and lie in
// shared memory as they do in memory; ldmatrix turns those stored along i or j. The
// next step's loads are under way while one is multiplied. Forward, dx, dW in us: 5120
// routes of 64 experts, 2559 -> 641, 429, 316, 398 (39 to 53 TFLOP/s); 8192 of 4 experts,
// 2049 -> 2047, 592, 597, 562 (116 to 122); element by element, in tiles of 64, it was 25
// to 30 TFLOP/s. Bound by the latency of those loads: two CTAs an SM, each one step
// ahead. One CTA an SM that holds raw words in registers: 353, 303, 491 and 646, 614,
// 696; the words by cp.async three steps ahead: 373, 308, 519 and 727, 691, 779.
constexpr int kGenTile = 128, kGenStep = 32, kGenThreads = 256;
constexpr int kGenAlong = kGenStep + 8, kGenAcross = kGenTile + 8;  // elements between rows in shared memory
constexpr int kGenBytes = kGenTile * kGenAlong * 2;                 // (the larger of the two layouts)

__device__ __forceinline__ void gen_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void gen_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool TRANS>
__device__ __forceinline__ void gen_ldmatrix(uint32_t (&r)[4], uint32_t at) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

// The memory that a tensor's rows and what lies between them take.
struct GenSpan {
  uintptr_t lo, hi;
};

// n (at most eight, none if below 1) elements of 16 bits at p, then zeros.
__device__ __forceinline__ uint4 gen_load8(const uint16_t* p, int n, GenSpan in) {
  uint4 q = make_uint4(0, 0, 0, 0);
  if (n <= 0) return q;
  const uintptr_t at = (uintptr_t)p, w0 = at & ~(uintptr_t)15;
  const int off = (int)(at & 15);
  const bool two = off + 2 * n > 16 && off;
  if (w0 >= in.lo && w0 + (two ? 32 : 16) <= in.hi) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(w0));
    const uint4 y = two ? __ldg(reinterpret_cast<const uint4*>(w0) + 1) : make_uint4(0, 0, 0, 0);
    // the eight words from byte `off` on, by 8, 4 and 2 bytes
    const bool e = off & 8, f = off & 4;
    const uint32_t a0 = e ? x.z : x.x, a1 = e ? x.w : x.y, a2 = e ? y.x : x.z, a3 = e ? y.y : x.w, a4 = e ? y.z : y.x, a5 = e ? y.w : y.y;
    const uint32_t b0 = f ? a1 : a0, b1 = f ? a2 : a1, b2 = f ? a3 : a2, b3 = f ? a4 : a3, b4 = f ? a5 : a4;
    const int s = (off & 2) * 8;
    q = make_uint4(__funnelshift_r(b0, b1, s), __funnelshift_r(b1, b2, s), __funnelshift_r(b2, b3, s), __funnelshift_r(b3, b4, s));
    if (n < 8) {
      auto keep = [&](uint32_t w, int i) { return n >= 2 * i + 2 ? w : n == 2 * i + 1 ? w & 0xFFFFu : 0u; };
      q = make_uint4(keep(q.x, 0), keep(q.y, 1), keep(q.z, 2), keep(q.w, 3));
    }
  } else {  // (the tensor's first and last words)
    uint32_t w[4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) w[i >> 1] |= (uint32_t)__ldg(p + i) << (16 * (i & 1));
    q = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return q;
}

template <typename T, typename O, int MODE>
__global__ void __launch_bounds__(kGenThreads, 2) k_ex_general(const ExArgs a) {
  __shared__ __align__(16) unsigned char s_tile[2][2][kGenBytes];  // by step, operand
  __shared__ int s_off[kExMaxExperts + 2], s_first[kExMaxExperts + 2], s_row[kGenTile];
  constexpr bool kAcrossA = MODE == kExGradW, kAcrossB = MODE != kExForward;  // stored along i, j
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
    if (tid < kGenTile) s_row[tid] = i0 + tid < I ? a.order[s_off[expert] + i0 + tid] : -1;
    __syncthreads();
  }
  const int j0 = blockIdx.y * kGenTile, base = s_off[expert];
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  const uint16_t* g = static_cast<const uint16_t*>(a.g);
  const uint16_t* wall = static_cast<const uint16_t*>(a.w);
  const uint16_t* w = wall + (size_t)(expert < E ? expert : 0) * a.lde;
  auto span = [](const uint16_t* p, int64_t last, int64_t ld, int cols) {
    return GenSpan{(uintptr_t)p, (uintptr_t)(p + last * ld + cols)};
  };
  const GenSpan xs = span(x, (a.per_route ? R : a.T) - 1, a.ldx, a.K), gs = span(g, R - 1, a.ldg, a.N);
  const GenSpan ws{(uintptr_t)wall, (uintptr_t)(wall + (int64_t)(E - 1) * a.lde + (int64_t)(a.N - 1) * a.ldw + a.K)};
  auto source = [&](int route) { return a.per_route ? route : route / a.topk; };
  // a thread's two pieces of each operand: along k, rows tid / 4 and 64 more, piece tid % 4;
  // across, steps tid / 16 and 16 more, piece tid % 16
  const int ar = tid >> 2, ac = (tid & 3) * 8, br = tid >> 4, bc = (tid & 15) * 8;
  uint4 qa[2], qb[2];
  int route[2];  // grad_w: of the step to be loaded
  auto look = [&](int k0) {
    if (MODE == kExGradW) {
#pragma unroll
      for (int u = 0; u < 2; ++u) route[u] = k0 + br + 16 * u < depth ? __ldg(a.order + base + k0 + br + 16 * u) : -1;
    }
  };
  auto load = [&](int k0) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (MODE == kExGradW) {
        const bool in = route[u] >= 0;
        qa[u] = gen_load8(g + (in ? (size_t)route[u] * a.ldg + i0 + bc : 0), in ? min(8, I - i0 - bc) : 0, gs);
        qb[u] = gen_load8(x + (in ? (size_t)source(route[u]) * a.ldx + j0 + bc : 0), in ? min(8, J - j0 - bc) : 0, xs);
      } else {
        const int r = s_row[ar + 64 * u], n = min(8, depth - k0 - ac), j = j0 + ar + 64 * u;
        if (MODE == kExForward) {
          qa[u] = gen_load8(x + (r >= 0 ? (size_t)source(r) * a.ldx + k0 + ac : 0), r >= 0 ? n : 0, xs);
          qb[u] = gen_load8(w + (j < J ? (size_t)j * a.ldw + k0 + ac : 0), j < J ? n : 0, ws);
        } else {
          const int k = k0 + br + 16 * u;
          qa[u] = gen_load8(g + (r >= 0 ? (size_t)r * a.ldg + k0 + ac : 0), r >= 0 ? n : 0, gs);
          qb[u] = gen_load8(w + (k < depth ? (size_t)k * a.ldw + j0 + bc : 0), k < depth ? min(8, J - j0 - bc) : 0, ws);
        }
      }
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int along = ((ar + 64 * u) * kGenAlong + ac) * 2, across = ((br + 16 * u) * kGenAcross + bc) * 2;
      *reinterpret_cast<uint4*>(s_tile[buf][0] + (kAcrossA ? across : along)) = qa[u];
      *reinterpret_cast<uint4*>(s_tile[buf][1] + (kAcrossB ? across : along)) = qb[u];
    }
  };
  float acc[4][4][4] = {};  // the warp's 64 x 32: rows of 16, columns of 8
  const int wi = (warp >> 2) * 64, wj = (warp & 3) * 32;
  const int steps = (depth + kGenStep - 1) / kGenStep;
  if (steps > 0) {
    look(0);
    load(0);
    look(kGenStep);
    put(0);
  }
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    if (s + 1 < steps) {
      load((s + 1) * kGenStep);
      look((s + 2) * kGenStep);
    }
    const uint32_t ta = (uint32_t)__cvta_generic_to_shared(s_tile[s & 1][0]), tb = (uint32_t)__cvta_generic_to_shared(s_tile[s & 1][1]);
#pragma unroll
    for (int kk = 0; kk < kGenStep; kk += 16) {
      uint32_t fa[4][4], fb[2][4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int i = wi + m * 16;
        if (kAcrossA)
          gen_ldmatrix<true>(fa[m], ta + ((kk + (lane & 7) + ((lane >> 4) << 3)) * kGenAcross + i + ((lane >> 3) & 1) * 8) * 2);
        else
          gen_ldmatrix<false>(fa[m], ta + ((i + (lane & 15)) * kGenAlong + kk + (lane >> 4) * 8) * 2);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int j = wj + n * 16;
        if (kAcrossB)
          gen_ldmatrix<true>(fb[n], tb + ((kk + (lane & 15)) * kGenAcross + j + (lane >> 4) * 8) * 2);
        else
          gen_ldmatrix<false>(fb[n], tb + ((j + (lane & 7) + ((lane >> 4) << 3)) * kGenAlong + kk + ((lane >> 3) & 1) * 8) * 2);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) gen_mma(acc[m][n], fa[m], fb[n >> 1][(n & 1) * 2], fb[n >> 1][(n & 1) * 2 + 1], T());
    }
    if (s + 1 < steps) put((s + 1) & 1);
    __syncthreads();
  }
  O* out = static_cast<O*>(a.out);
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = wi + m * 16 + (lane >> 2) + h * 8;
      if (i0 + i >= I) continue;
      O* row = out + (MODE == kExGradW ? (size_t)expert * a.N + i0 + i : (size_t)s_row[i]) * J;
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int j = j0 + wj + n * 8 + (lane & 3) * 2 + v;
          if (j < J) row[j] = from_f32<O>(acc[m][n][2 * h + v]);
        }
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
