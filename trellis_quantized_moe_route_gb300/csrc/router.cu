// Router with load statistics and losses, and its gradient (sm_103a).
//
// For logits l [T, E] with p = softmax(l) over the experts and S_t the k
// largest logits of token t (ties to the lowest id):
//   w_tj  = exp(l_t,id_j) / sum_i exp(l_t,id_i)      the layer's route weights
//   lse_t = log sum_e exp(l_te)
// Over the n valid tokens (mask set, and some logit above -inf):
//   counts_e = routes to e whose logit is above -inf,  f_e = counts_e / (n k)
//   prob_e   = (1/n) sum_t p_te
//   losses   = { E sum_e f_e prob_e,  (1/n) sum_t lse_t^2 }
// Gradient, counts held constant, for upstream g_b, g_z and dw [T, k]:
//   dl_te = p_te ((g_b E/n)(f_e - sum_e' f_e' p_te') + (2 g_z/n) lse_t)   valid tokens
//         + w_tj (dw_tj - sum_i w_ti dw_ti)                              e = id_j
// All of it in fp32 whatever the logits' type; only dl is rounded to it.
//
// One warp takes a token, V logits a lane, and reads the next token's row while
// it works on this one (many tokens of 16-bit logits: a lane a token, below).
// The selection's instructions and their latency bound it, not the bytes. Each
// logit becomes a 32-bit key that is unique in the row and orders
// like (logit, then lower expert): 16-bit logits have their expert in the low
// half; fp32 logits give up their lowest 8 bits for it, and a token in which two
// of the k + 1 largest agree in the other 24 (one in a few hundred, or equal
// logits) is selected again on the whole values. A lane sorts its keys once
// (min / max only, nothing carried along); each of the k rounds is then one
// warp-wide maximum of the lanes' first keys, and the lane that held it moves up.
//
// Probability sums stay in registers over all of a warp's tokens, are added over
// the CTA's warps and the cluster's CTAs in shared memory and over the clusters
// by a second kernel (with up to 128 tokens there is one cluster and no second
// kernel), always in the same order; counts are integers. So the same bits every
// time. The backward pass reads the logits again and rebuilds p from lse, which
// costs less than storing p (T E fp32).
//
// Exponentials, the logarithm and the quotients are the hardware's approximations
// of 2 ulp or so: beside the arguments' rounding in fp32 they add little (w, prob
// and lse are off by 1e-7 of themselves); the logarithm's error is absolute, so
// that an lse near 0 has fewer right bits.
//
// 65536 tokens x 160 bf16 logits, k = 8, masked: forward 16 us with a lane a token
// (160 instructions a token; its bytes take 4 us; with a warp a token 24: 360
// instructions), finishing sums 5 us, backward 15.4 us (220 instructions a token;
// its bytes take 7 us). Both are bound by latency: the forward kernel issues in
// 36% of its cycles (integer pipe 41% busy, DRAM 12%), since a group's rows are
// waited for with nothing of the next one under way; the backward kernel in 52%
// (42%, 16%), with 4 bytes a lane and load. fp32 logits, all a warp a token:
// forward 35 us, backward 18.6 us. 8 tokens x 128: one launch, 3.1 us.
#include <algorithm>

#include "elem.cuh"
#include "pdl.cuh"
#include "status.h"

namespace tmoe {

namespace {

constexpr int kRtWarps = 16;      // warps of a CTA with many tokens
constexpr int kRtBwdCtas = 5;         // CTAs of 256 threads that an SM holds of the backward kernel
constexpr int kRtMaxClusters = 152;  // of two CTAs each: two CTAs of 512 threads on each of 152 SMs

// Orderable bits of a logit (larger value, larger bits; -0 as +0), in the upper
// bits of a word, and back. kNone: the largest such word for -inf. Every key is
// made after an addition of +0, here or in add_zero: it turns -0 into +0 and a
// NaN of either sign into the positive one, whose key is above all others. So
// nothing in a row lies below -inf, and no absent expert before a real one.
template <typename T>
struct Order;
template <>
struct Order<float> {
  static constexpr uint32_t kMask = 0xFFFFFF00u, kNone = 0x007FFFFFu;
  static __device__ __forceinline__ uint32_t key(float f) {
    const uint32_t b = __float_as_uint(f + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
  }
};
// (16-bit types: `bits` has the logit in its upper half, zeros below)
struct Order16 {
  static constexpr uint32_t kMask = 0xFFFF0000u;
  static __device__ __forceinline__ uint32_t key(uint32_t bits) {
    return bits ^ (((uint32_t)((int32_t)bits >> 31) & 0x7FFF0000u) | 0x80000000u);
  }
};
template <>
struct Order<__nv_bfloat16> : Order16 {
  static constexpr uint32_t kNone = 0x007FFFFFu;  // -inf is 0xFF80
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xFFFF0000u));
  }
};
template <>
struct Order<__half> : Order16 {
  static constexpr uint32_t kNone = 0x03FFFFFFu;  // -inf is 0xFC00
  static __device__ __forceinline__ float value(uint32_t k) {
    return __half2float(__ushort_as_half((unsigned short)((k ^ ((k & 0x80000000u) ? 0x80000000u : 0xFFFF0000u)) >> 16)));
  }
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ int cluster_peer(const int* p, int rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];\n" : "=r"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// exp(x) for x <= 0 or NaN by the hardware's exp2 (the product's rounding is
// |x| 2^-24, as the subtraction's before it).
__device__ __forceinline__ float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}

// The sum over the first k lanes' values in all of them (others hold 0); a
// warp-wide sum where k > 8.
__device__ __forceinline__ float first_sum(float v, int k) {
  if (k > 8) {
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// A row of logits over a warp: V of them a lane (V even). 16-bit types take
// neighbours in pairs, one 4-byte load each with PAIR (an even number of experts,
// rows 4 bytes aligned). Past the
// last expert stands -inf: with a higher number than any expert, it comes after
// an expert's own -inf, and its probability is 0.
template <int V, typename T, bool PAIR>
struct RowRegs {
  uint32_t raw[sizeof(T) == 2 ? V / 2 : V];

  static __device__ __forceinline__ int expert(int i) {
    const int lane = threadIdx.x & 31;
    return sizeof(T) == 2 ? 2 * lane + 64 * (i >> 1) + (i & 1) : lane + 32 * i;
  }
  static constexpr uint32_t kInf16 = sizeof(T) == 2 ? Order<T>::kNone >> 16 : 0;  // ~ of -inf's bits
  __device__ __forceinline__ void load(const T* __restrict__ row, int E) {
    if (sizeof(T) == 2) {
      const uint32_t none = 0xFFFFu & ~kInf16;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const int e = expert(2 * i);
        const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + e;
        raw[i] = none | none << 16;
        if (PAIR) {
          if (e < E) raw[i] = __ldg(reinterpret_cast<const uint32_t*>(p));
        } else if (e < E) {
          raw[i] = __ldg(p) | (e + 1 < E ? (uint32_t)__ldg(p + 1) : none) << 16;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        raw[i] = 0xFF800000u;
        if (expert(i) < E) raw[i] = __ldg(reinterpret_cast<const uint32_t*>(row) + expert(i));
      }
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if (sizeof(T) == 4) return __uint_as_float(raw[i]);
    if (std::is_same<T, __nv_bfloat16>::value)
      return __uint_as_float(i & 1 ? raw[i >> 1] & 0xFFFF0000u : raw[i >> 1] << 16);
    const uint16_t h = (uint16_t)(raw[i >> 1] >> (16 * (i & 1)));
    return to_f32(*reinterpret_cast<const T*>(&h));
  }
  // The row's largest logit, NaN if there is one (fp32). Beside the selection, so
  // that the probabilities need not wait for it: with the first selected one read
  // again in its place, 8 x 128 takes 3.3 us instead of 3.1, and 65536 x 160
  // 34.5 instead of 35.0.
  __device__ __forceinline__ float largest() const {
    uint32_t k = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) k = max(k, Order<float>::key(__uint_as_float(raw[i])));
    return Order<float>::value(__reduce_max_sync(0xFFFFFFFFu, k));
  }
  // Unique keys: the logit's order, then the lower expert.
  __device__ __forceinline__ void keys(uint32_t (&key)[V]) const {
    if (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        key[i] = (Order<float>::key(__uint_as_float(raw[i])) & Order<T>::kMask) | (0xFFu - (uint32_t)expert(i));
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const uint32_t w = add_zero(raw[i]);
        key[2 * i] = Order16::key(w << 16) | (0xFFFFu - (uint32_t)expert(2 * i));
        key[2 * i + 1] = Order16::key(w & 0xFFFF0000u) | (0xFFFFu - (uint32_t)expert(2 * i + 1));
      }
    }
  }
  // -0 becomes +0, a NaN the positive one (see Order)
  static __device__ __forceinline__ uint32_t add_zero(uint32_t w) {
    if (std::is_same<T, __nv_bfloat16>::value) {
      const __nv_bfloat162 s = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(0.0f));
      return *reinterpret_cast<const uint32_t*>(&s);
    }
    const __half2 s = __hadd2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(0.0f));
    return *reinterpret_cast<const uint32_t*>(&s);
  }
};

struct RouterFwd {
  const void* logits;
  int64_t ld;
  const uint8_t* mask;
  int T, E, k;
  int32_t* ids;
  float* w;
  float* lse;
  int32_t* counts;
  float* prob;
  float* losses;
  int32_t* tokens;
  // per cluster: [E] probability sums, [E] counts, then sum lse^2 and valid tokens
  float* part_prob;
  int32_t* part_counts;
  float* part_z;
  int32_t* part_n;
};

// Writes the results from sums over all tokens: thread e < E brings its
// expert's, every thread z and n.
__device__ __forceinline__ void router_write(const RouterFwd& a, float p, int c, float z, int n) {
  __shared__ float s_dot[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float inv_n = n > 0 ? 1.0f / (float)n : 0.0f;
  float dot = 0.0f;
  if (tid < a.E) {
    p *= inv_n;
    a.prob[tid] = p;
    a.counts[tid] = c;
    dot = (float)c * inv_n / (float)a.k * p;
  }
  dot = warp_sum(dot);
  if (lane == 0) s_dot[warp] = dot;
  __syncthreads();
  if (warp == 0) {
    dot = warp_sum(lane < (int)(blockDim.x >> 5) ? s_dot[lane] : 0.0f);
    if (lane == 0) {
      a.losses[0] = (float)a.E * dot;
      a.losses[1] = z * inv_n;
      *a.tokens = n;
    }
  }
}

// Adds up the clusters' statistics, by one cluster of kFinCtas CTAs: CTA q the
// parts q, q + kFinCtas, ... in order (its loads all in flight), then the first
// CTA the CTAs' sums in rank order.
constexpr int kFinCtas = 8;

__global__ void __cluster_dims__(kFinCtas, 1, 1) __launch_bounds__(kMaxExperts) k_router_finish(RouterFwd a, int parts) {
  constexpr int kEach = (kRtMaxClusters + kFinCtas - 1) / kFinCtas;
  __shared__ float s_p[kMaxExperts], s_z;
  __shared__ int s_c[kMaxExperts], s_n;
  const int e = threadIdx.x, q = (int)cluster_rank();
  grid_wait();
  grid_launch();
  float p[kEach], z[kEach];
  int c[kEach], n[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int u = q + kFinCtas * i;
    p[i] = u < parts && e < a.E ? a.part_prob[u * a.E + e] : 0.0f;
    c[i] = u < parts && e < a.E ? a.part_counts[u * a.E + e] : 0;
    z[i] = u < parts ? a.part_z[u] : 0.0f;
    n[i] = u < parts ? a.part_n[u] : 0;
  }
#pragma unroll
  for (int i = 1; i < kEach; ++i) {
    p[0] += p[i];
    c[0] += c[i];
    z[0] += z[i];
    n[0] += n[i];
  }
  s_p[e] = p[0];
  s_c[e] = c[0];
  if (e == 0) {
    s_z = z[0];
    s_n = n[0];
  }
  cluster_sync();
  if (q == 0) {
    float pp = 0.0f, zz = 0.0f;
    int cc = 0, nn = 0;
#pragma unroll
    for (int u = 0; u < kFinCtas; ++u) {
      pp += __int_as_float(cluster_peer(reinterpret_cast<const int*>(&s_p[e]), u));
      cc += cluster_peer(&s_c[e], u);
      zz += __int_as_float(cluster_peer(reinterpret_cast<const int*>(&s_z), u));
      nn += cluster_peer(&s_n, u);
    }
    router_write(a, pp, cc, zz, nn);
  }
  cluster_sync();  // no CTA leaves while its sums are read
}

// The k largest of a row: lane j < k returns the j-th expert. `key`: the unique
// keys (0: absent), consumed. Returns whether the order is certain.
template <int V, typename T>
__device__ __forceinline__ bool router_select(uint32_t (&key)[V], int k, int E, uint32_t& mine, uint32_t& first) {
  const int lane = threadIdx.x & 31;
  // odd-even transposition, largest first
#pragma unroll
  for (int r = 0; r < V; ++r)
#pragma unroll
    for (int i = r & 1; i + 1 < V; i += 2) {
      const uint32_t hi = max(key[i], key[i + 1]);
      key[i + 1] = min(key[i], key[i + 1]);
      key[i] = hi;
    }
  const int rounds = sizeof(T) == 4 && k < E ? k + 1 : k;  // (fp32: the first one left out, too)
  uint32_t extra = 0;
  auto round = [&] {
    const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, key[0]);
    if (key[0] == best) {
#pragma unroll
      for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
      key[V - 1] = 0u;
    }
    return best;
  };
  mine = first = round();
#pragma unroll 4
  for (int j = 1; j < rounds; ++j) {
    extra = round();  // (k = 32: the last one is in no lane)
    if (lane == j) mine = extra;
  }
  if (sizeof(T) == 2) return true;
  uint32_t next = __shfl_down_sync(0xFFFFFFFFu, mine, 1);
  if (lane == 31) next = extra;
  const bool same = lane + 1 < rounds && ((mine ^ next) & Order<T>::kMask) == 0;
  return !__any_sync(0xFFFFFFFFu, same);
}

// The same on the whole fp32 values, equal ones by the lower expert.
template <int V>
__device__ __noinline__ uint32_t router_select_exact(const float* __restrict__ row, int k, int E) {
  const int lane = threadIdx.x & 31;
  uint32_t key[V], mine = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = lane + 32 * i < E ? Order<float>::key(row[lane + 32 * i]) : 0u;
  for (int j = 0; j < k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = max(m, key[i]);
    const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, m);
    uint32_t id = 0xFFFFFFFFu;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (key[i] == best) id = lane + 32 * i;
    id = __reduce_min_sync(0xFFFFFFFFu, id);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i == (int)id) key[i] = 0u;
    if (lane == j) mine = id;
  }
  return mine;
}

// Adds up a CTA's statistics (s_acc: its warps' probability sums, `width` floats
// apart; s_z, s_nv: theirs too; s_cnt: the CTA's), then its cluster's of csize
// CTAs. With one cluster the results are written here, with more its part.
__device__ __forceinline__ void router_stats(const RouterFwd& a, int csize, int rank, int warps, float* s_acc,
                                             int width, int* s_cnt, float* s_z, int* s_nv) {
  // the CTA's sums, in warp order
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    float p = 0.0f;
    for (int u = 0; u < warps; ++u) p += s_acc[u * width + e];
    s_acc[e] = p;
  }
  if (threadIdx.x == 0) {
    for (int u = 1; u < warps; ++u) {
      s_z[0] += s_z[u];
      s_nv[0] += s_nv[u];
    }
  }
  // the cluster's, in rank order, by its first CTA
  float p = 0.0f, zs = 0.0f;
  int c = 0, ns = 0;
  const int e = threadIdx.x;
  if (csize > 1) {
    cluster_sync();
    if (rank == 0) {
      for (int u = 0; u < csize; ++u) {
        if (e < a.E) {
          p += __int_as_float(cluster_peer(reinterpret_cast<const int*>(&s_acc[e]), u));
          c += cluster_peer(&s_cnt[e], u);
        }
        zs += __int_as_float(cluster_peer(reinterpret_cast<const int*>(&s_z[0]), u));
        ns += cluster_peer(&s_nv[0], u);
      }
    }
    cluster_sync();  // no CTA leaves while its sums are read
    if (rank != 0) return;
  } else {
    __syncthreads();
    if (e < a.E) {
      p = s_acc[e];
      c = s_cnt[e];
    }
    zs = s_z[0];
    ns = s_nv[0];
  }
  if ((int)gridDim.x == csize) {
    router_write(a, p, c, zs, ns);
  } else {
    const int part = blockIdx.x / csize;
    if (e < a.E) {
      a.part_prob[part * a.E + e] = p;
      a.part_counts[part * a.E + e] = c;
    }
    if (e == 0) {
      a.part_z[part] = zs;
      a.part_n[part] = ns;
    }
  }
}

// A warp's tokens are warp, warp + W, ... (W: warps of the grid). With one
// cluster (of csize CTAs) the statistics are finished here.
template <int V, typename T, bool PAIR>
__global__ void __launch_bounds__(kRtWarps * 32, 2) k_router_fwd(RouterFwd a, int csize) {
  using Row = RowRegs<V, T, PAIR>;
  __shared__ float s_acc[kRtWarps][V * 32];
  __shared__ int s_cnt[V * 32];
  __shared__ float s_z[kRtWarps];
  __shared__ int s_nv[kRtWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int rank = csize > 1 ? (int)cluster_rank() : 0;
  grid_wait();
  grid_launch();
  for (int e = threadIdx.x; e < V * 32; e += blockDim.x) s_cnt[e] = 0;
  __syncthreads();
  const T* logits = static_cast<const T*>(a.logits);
  float acc[V] = {};
  float z = 0.0f;
  int n = 0;
  const int step = gridDim.x * warps;
  int t = blockIdx.x * warps + warp;
  Row row;
  if (t < a.T) row.load(logits + (size_t)t * a.ld, a.E);
  for (; t < a.T; t += step) {
    const Row now = row;
    if (t + step < a.T) row.load(logits + (size_t)(t + step) * a.ld, a.E);
    const bool on = a.mask == nullptr || a.mask[t] != 0;
    uint32_t key[V], mine, first;
    now.keys(key);
    const bool sure = router_select<V, T>(key, a.k, a.E, mine, first);
    uint32_t id = ~Order<T>::kMask - (mine & ~Order<T>::kMask);
    const T* src = logits + (size_t)t * a.ld;
    if (sizeof(T) == 4 && !sure) id = router_select_exact<V>(reinterpret_cast<const float*>(src), a.k, a.E);
    // The softmax's offset is the row's largest logit to the last bit: fp32's key
    // lacks the low ones, which are worth thousands where logits are of 1e9.
    const bool some = first > Order<T>::kNone;
    const float m = sizeof(T) == 4 ? now.largest() : Order<T>::value(first & Order<T>::kMask);
    float my_l = 0.0f;
    if (lane < a.k) my_l = sizeof(T) == 4 ? to_f32(src[id]) : Order<T>::value(mine & Order<T>::kMask);
    float p[V], total = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = exp_fast(now.get(i) - m);
      total += p[i];
    }
    total = warp_sum(total);
    const float we = lane < a.k ? exp_fast(my_l - m) : 0.0f;
    const float wsum = first_sum(we, a.k);
    const float lse = m + __logf(total);
    if (lane < a.k) {
      a.ids[(size_t)t * a.k + lane] = (int)id;
      a.w[(size_t)t * a.k + lane] = some ? __fdividef(we, wsum) : 0.0f;
      if (on && some && my_l != -INFINITY) atomicAdd(&s_cnt[id], 1);
    }
    if (lane == 0) a.lse[t] = some ? lse : -INFINITY;
    if (on && some) {
      const float inv = __fdividef(1.0f, total);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += p[i] * inv;
      z += lse * lse;
      ++n;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) s_acc[warp][Row::expert(i)] = acc[i];
  if (lane == 0) {
    s_z[warp] = z;
    s_nv[warp] = n;
  }
  __syncthreads();
  router_stats(a, csize, rank, warps, &s_acc[0][0], V * 32, s_cnt, s_z, s_nv);
}

// The same for many tokens of 16-bit logits and k <= 8, a lane a token: a warp
// brings 32 rows to shared memory, and each lane finds the k largest of one of
// them with a list of the eight largest so far, eight keys at a time: sorted by
// a network of 19 exchanges, merged by eight maxima and 12 exchanges more.
// Probabilities are made with a warp's lanes over the experts again, since their
// sums go over the tokens. Rows lie an odd number of 16 bytes apart, so that
// neither way of reading meets bank conflicts. 160 instructions a token with 160
// experts, where a warp a token takes 360. At 65536 tokens an SM has 13.5 of
// these groups of 32, and a quarter of it (one scheduler) 3 or 4, each of which
// waits for its own rows before it starts: of the 16 us, 3.3 for each of the four,
// and the rest is the statistics.
constexpr int kRtLaneWarps = 8;

__device__ __forceinline__ void exchange(int32_t& a, int32_t& b) {
  const int32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}

template <int V, typename T>
__global__ void __launch_bounds__(kRtLaneWarps * 32, 2) k_router_fwd_lanes(RouterFwd a, int csize, FastDiv units) {
  using Row = RowRegs<V, T, true>;
  extern __shared__ uint4 s_rows[];
  __shared__ int s_cnt[V * 32];
  __shared__ float s_z[kRtLaneWarps];
  __shared__ int s_nv[kRtLaneWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = csize > 1 ? (int)cluster_rank() : 0;
  const int nu = (int)units.d, pitch = nu | 1;
  uint4* rows = s_rows + (size_t)warp * 32 * pitch;
  grid_wait();
  grid_launch();
  for (int e = threadIdx.x; e < V * 32; e += blockDim.x) s_cnt[e] = 0;
  __syncthreads();
  const T* logits = static_cast<const T*>(a.logits);
  float acc[V] = {};
  float z = 0.0f;
  int n = 0;
  const int groups = (a.T + 31) / 32;
  for (int g = warp * (int)gridDim.x + (int)blockIdx.x; g < groups; g += (int)gridDim.x * kRtLaneWarps) {
    const int t0 = g * 32, count = min(32, a.T - t0);
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(rows);
    for (int i = lane; i < count * nu; i += 32) {
      const int r = (int)units.div(i), c = i - r * nu;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to + (uint32_t)(r * pitch + c) * 16u),
                   "l"(logits + (size_t)(t0 + r) * a.ld + c * 8)
                   : "memory");
    }
    const bool in = lane < count;
    const bool on = in && (a.mask == nullptr || a.mask[t0 + lane] != 0);
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    __syncwarp();
    // keys as above, in signed order; `low` has the experts' part for two of them
    uint32_t low[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) low[i] = (0xFFFFu - 2u * i) | (0xFFFEu - 2u * i) << 16;
    auto read = [&](int c, int32_t(&key)[8]) {
      const uint4 q = rows[lane * pitch + c];
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t v = Row::add_zero(w[i]), sign;
        asm("prmt.b32 %0, %1, %1, 0xBB99;" : "=r"(sign) : "r"(v));  // each half's sign in all its bits
        v ^= sign & 0x7FFF7FFFu;
        key[2 * i] = (int32_t)__byte_perm(v, low[i], 0x1054);
        key[2 * i + 1] = (int32_t)__byte_perm(v, low[i], 0x3276);
        low[i] -= 0x00080008u;
      }
      exchange(key[0], key[1]), exchange(key[2], key[3]), exchange(key[4], key[5]), exchange(key[6], key[7]);
      exchange(key[0], key[2]), exchange(key[1], key[3]), exchange(key[4], key[6]), exchange(key[5], key[7]);
      exchange(key[1], key[2]), exchange(key[5], key[6]);
      exchange(key[0], key[4]), exchange(key[1], key[5]), exchange(key[2], key[6]), exchange(key[3], key[7]);
      exchange(key[2], key[4]), exchange(key[3], key[5]);
      exchange(key[1], key[2]), exchange(key[3], key[4]), exchange(key[5], key[6]);
    };
    int32_t top[8];
    read(0, top);
#pragma unroll 2
    for (int c = 1; c < nu; ++c) {
      int32_t key[8];
      read(c, key);
#pragma unroll
      for (int i = 0; i < 8; ++i) top[i] = max(top[i], key[7 - i]);
#pragma unroll
      for (int d = 4; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!(i & d)) exchange(top[i], top[i + d]);
    }
    const auto value = [](int32_t key) { return Order<T>::value(((uint32_t)key ^ 0x80000000u) & Order<T>::kMask); };
    const bool some = ((uint32_t)top[0] ^ 0x80000000u) > Order<T>::kNone;
    const float m = value(top[0]);
    const bool valid = on && some;
    {
      float we[8], sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        we[j] = j < a.k ? exp_fast(value(top[j]) - m) : 0.0f;
        sum += we[j];
      }
      int32_t* ids = a.ids + (size_t)(t0 + lane) * a.k;
      float* w = a.w + (size_t)(t0 + lane) * a.k;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < a.k && in) {
          const int id = 0xFFFF - (top[j] & 0xFFFF);
          ids[j] = id;
          w[j] = some ? __fdividef(we[j], sum) : 0.0f;
          if (valid && value(top[j]) != -INFINITY) atomicAdd(&s_cnt[id], 1);
        }
      }
    }
    const uint32_t valids = __ballot_sync(0xFFFFFFFFu, valid);
    // Four tokens at a time: their sums over the lanes are folded into one value,
    // the lanes' upper two bits saying whose it is.
    float mine = 0.0f;
    const bool hi = lane & 16, mid = lane & 8;
#pragma unroll 1
    for (int t = 0; t < count; t += 4) {  // (rows past the last are there, too, and count for nothing)
      float p[4][V], total[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        Row row;
        const uint32_t* words = reinterpret_cast<const uint32_t*>(rows + (t + j) * pitch);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const uint32_t none = 0xFFFFu & ~Row::kInf16;
          row.raw[i] = none | none << 16;
          if (Row::expert(2 * i) < a.E) row.raw[i] = words[lane + 32 * i];
        }
        const float mt = __shfl_sync(0xFFFFFFFFu, m, t + j);
        total[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          p[j][i] = exp_fast(row.get(i) - mt);
          total[j] += p[j][i];
        }
      }
      const float x0 = __shfl_xor_sync(0xFFFFFFFFu, hi ? total[0] : total[2], 16);
      const float x1 = __shfl_xor_sync(0xFFFFFFFFu, hi ? total[1] : total[3], 16);
      const float u0 = (hi ? total[2] : total[0]) + x0, u1 = (hi ? total[3] : total[1]) + x1;
      float v = (mid ? u1 : u0) + __shfl_xor_sync(0xFFFFFFFFu, mid ? u0 : u1, 8);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      const float of = __shfl_sync(0xFFFFFFFFu, v, (lane & 3) * 8);
      if (lane >> 2 == t >> 2) mine = of;
      const float inv = __fdividef(1.0f, v);
      float f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = __shfl_sync(0xFFFFFFFFu, inv, j * 8);
      const uint32_t four = valids >> t & 15;
      if (four == 15) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] += p[j][i] * f[j];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (four >> j & 1)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += p[j][i] * f[j];
      }
    }
    if (in) {
      const float lse = m + __logf(mine);
      a.lse[t0 + lane] = some ? lse : -INFINITY;
      if (valid) z += lse * lse;
    }
    n += __popc(valids);
    __syncwarp();  // (the rows are read before the next ones come)
  }
  z = warp_sum(z);
  __syncthreads();
  float* s_acc = reinterpret_cast<float*>(s_rows);  // (at least as large: 16 bytes a lane and unit)
#pragma unroll
  for (int i = 0; i < V; ++i) s_acc[warp * V * 32 + Row::expert(i)] = acc[i];
  if (lane == 0) {
    s_z[warp] = z;
    s_nv[warp] = n;
  }
  __syncthreads();
  router_stats(a, csize, rank, kRtLaneWarps, s_acc, V * 32, s_cnt, s_z, s_nv);
}

struct RouterBwd {
  const void* logits;
  int64_t ld;
  const uint8_t* mask;
  int T, E, k;
  const int32_t* ids;
  const float* w;
  const float* lse;
  const int32_t* counts;
  const int32_t* tokens;
  const float* grad_w;       // [T, k] or NULL
  const float* grad_losses;  // [2] or NULL
  void* grad_logits;         // [T, E]
};

template <int V, typename T, bool PAIR>
__global__ void __launch_bounds__(256, kRtBwdCtas) k_router_bwd(RouterBwd a) {
  using Row = RowRegs<V, T, PAIR>;
  __shared__ float s_sel[8][V * 32];  // each warp's selected experts' gradients, zero between tokens
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* logits = static_cast<const T*>(a.logits);
  T* grad = static_cast<T*>(a.grad_logits);
  grid_wait();
  grid_launch();
  const int n = *a.tokens;
  const float inv_n = n > 0 ? 1.0f / (float)n : 0.0f;
  const float gb = a.grad_losses ? a.grad_losses[0] * (float)a.E * inv_n : 0.0f;
  const float gz = a.grad_losses ? a.grad_losses[1] * 2.0f * inv_n : 0.0f;
  float f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = Row::expert(i);
    f[i] = e < a.E ? (float)a.counts[e] * inv_n / (float)a.k : 0.0f;
    s_sel[warp][lane + 32 * i] = 0.0f;
  }
  __syncwarp();
  // a token's inputs, read while the one before it is worked on
  struct In {
    Row row;
    float lse, w, g;
    int id;
    bool on;
  };
  auto read = [&](int t, In& in) {
    in.row.load(logits + (size_t)t * a.ld, a.E);
    in.lse = a.lse[t];
    in.on = a.mask == nullptr || a.mask[t] != 0;
    in.id = -1;
    in.w = in.g = 0.0f;
    if (a.grad_w && lane < a.k) {
      in.id = a.ids[(size_t)t * a.k + lane];
      in.w = a.w[(size_t)t * a.k + lane];
      in.g = a.grad_w[(size_t)t * a.k + lane];
    }
  };
  const int step = gridDim.x * 8;
  int t = blockIdx.x * 8 + warp;
  In next;
  if (t < a.T) read(t, next);
  for (; t < a.T; t += step) {
    const In in = next;
    if (t + step < a.T) read(t + step, next);
    const bool on = in.on && in.lse != -INFINITY;
    float p[V], s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = on ? exp_fast(in.row.get(i) - in.lse) : 0.0f;
      s += f[i] * p[i];
    }
    s = warp_sum(s);
    // lse is rounded, which makes all of p wrong by one factor: up to 1 + |lse|
    // 2^-24, and as much as the number of the logits where these are so large that
    // its logarithm is lost in lse. Their sum, which should be 1, takes it out
    // where that is above the exponents' own rounding (fp32) or an eighth of the
    // result's (16 bits: lse is within 2^-15 up to 1024). 65536 x 160 bf16: 15.5
    // us, with the sum for every token 16.9, and with the warp not known to agree
    // (no vote) 15.9.
    if (__any_sync(0xFFFFFFFFu, on && fabsf(in.lse) > (sizeof(T) == 4 ? 16.0f : 1024.0f))) {
      float total = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) total += p[i];
      const float r = __fdividef(1.0f, warp_sum(total));
      s *= r;
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] *= r;
    }
    const int id = in.id >= 0 && in.id < a.E ? in.id : -1;
    if (a.grad_w) {
      // (a weight of zero gets no gradient whatever comes from above, and a
      // zero from above gives none whatever the weight: padding may hold NaN)
      const float wg = in.w != 0.0f && in.g != 0.0f ? in.w * in.g : 0.0f;
      const float dot = first_sum(wg, a.k);
      if (id >= 0) s_sel[warp][id] = in.w != 0.0f && dot != 0.0f ? wg - in.w * dot : wg;
      __syncwarp();
    }
    const float c = gz * (on ? in.lse : 0.0f);
    T* out = grad + (size_t)t * a.E;
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = p[i] * (gb * (f[i] - s) + c) + s_sel[warp][Row::expert(i)];
    if (PAIR) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        uint32_t w;
        reinterpret_cast<T*>(&w)[0] = from_f32<T>(d[i]);
        reinterpret_cast<T*>(&w)[1] = from_f32<T>(d[i + 1]);
        if (Row::expert(i) < a.E) *reinterpret_cast<uint32_t*>(out + Row::expert(i)) = w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (Row::expert(i) < a.E) out[Row::expert(i)] = from_f32<T>(d[i]);
    }
    if (a.grad_w) {
      __syncwarp();
      if (id >= 0) s_sel[warp][id] = 0.0f;
      __syncwarp();
    }
  }
}

// Calls f with the number of logits a lane holds.
template <typename F>
cudaError_t by_width(int E, F f) {
  switch ((E + 63) / 64) {
    case 1: return f(std::integral_constant<int, 2>());
    case 2: return f(std::integral_constant<int, 4>());
    case 3: return f(std::integral_constant<int, 6>());
    default: return f(std::integral_constant<int, 8>());
  }
}

// Calls f with the logits' type and whether they can be taken in pairs.
template <typename F>
cudaError_t by_pairs(int32_t dtype, int E, const void* p, int64_t ld, const void* q, F f) {
  const bool pair = E % 2 == 0 && ((uintptr_t)p) % 4 == 0 && ld % 2 == 0 && ((uintptr_t)q) % 4 == 0;
  if (dtype == TM_F32) return f(float(), std::false_type());
  if (dtype == TM_BF16) return pair ? f(__nv_bfloat16(), std::true_type()) : f(__nv_bfloat16(), std::false_type());
  return pair ? f(__half(), std::true_type()) : f(__half(), std::false_type());
}

// CTAs of a cluster and clusters of a call: up to 128 tokens one cluster, which
// writes the results itself (one launch), then pairs (clusters of four do not
// fill the SMs: 64k tokens took 66 us forward and backward, with pairs 54 us).
struct RouterGrid {
  int csize, clusters;
};

RouterGrid router_grid(int T) {
  const int ctas = std::max(1, (T + kRtWarps - 1) / kRtWarps);
  if (ctas <= 8) {
    int c = 1;
    while (c < ctas) c *= 2;
    return {c, 1};
  }
  return {2, std::min(kRtMaxClusters, (ctas + 1) / 2)};
}

// Whether a call takes a lane a token: 16-bit logits in whole 16-byte pieces, at
// most the eight of its list, and tokens enough for the SMs' warps, 32 to each.
// us a forward call (bf16, masked), a warp / a lane a token:
//   tokens               20480         32768         49152         65536         200000
//   8 experts, k = 1     9.8 / 9.3     11.9 / 9.2    14.4 / 10.3   16.9 / 10.8   38 / 19
//   8 experts, k = 8     11.3 / 10.3   14.4 / 11.3   18.0 / 13.8   21.6 / 15.4   54 / 30
//   64 experts, k = 1    9.8 / 11.3    11.9 / 11.8   14.4 / 13.8   16.8 / 14.5   37 / 29
//   64 experts, k = 8    11.8 / 11.4   14.4 / 12.3   18.2 / 14.9   21.6 / 16.4   53 / 36
//   128 experts, k = 1   10.8 / 14.4   13.4 / 14.5   16.7 / 19.0   19.6 / 20.5   47 / 45
//   128 experts, k = 4   11.8 / 14.2   14.4 / 14.4   18.0 / 19.1   21.6 / 20.6   53 / 46
//   128 experts, k = 8   13.0 / 14.9   16.3 / 14.9   20.6 / 19.5   25.2 / 21.6   63 / 50
//   160 experts, k = 1   12.8 / 13.9   15.0 / 14.4   19.5 / 19.4   23.5 / 20.0   58 / 44
//   160 experts, k = 8   14.4 / 14.4   18.5 / 14.9   24.0 / 20.1   29.0 / 21.6   74 / 49
//   256 experts, k = 1   13.9 / 16.4   18.0 / 16.9   23.1 / 24.1   27.9 / 27.7   72 / 70
//   256 experts, k = 8   16.1 / 17.0   21.6 / 18.0   28.2 / 26.4   34.4 / 29.9   92 / 79
// The one limit on tokens is where most of these are even or better; with 128
// experts and k below 8 it comes too early (14% at the worst, 49152 tokens, k = 1),
// and a limit that moved with k would lose as much with 8, 64 and 160 experts.
constexpr int kRtLaneTokens = 32768;

bool router_lanes(const RouterFwd& a, int32_t dtype) {
  return dtype != TM_F32 && a.k <= 8 && a.T >= kRtLaneTokens && a.E % 8 == 0 && a.ld % 8 == 0 &&
         ((uintptr_t)a.logits) % 16 == 0;
}

template <int V, typename T>
cudaError_t router_lanes_launch(const RouterFwd& a, cudaLaunchConfig_t cfg, int csize) {
  auto kern = k_router_fwd_lanes<V, T>;
  constexpr int kMost = kRtLaneWarps * 32 * 16 * (kMaxExperts / 8 | 1);
  static OncePerDevice done;
  const cudaError_t limit = allow_smem(done, kern, kMost);
  if (limit != cudaSuccess) return limit;
  cfg.blockDim = dim3(32 * kRtLaneWarps);
  cfg.dynamicSmemBytes = (size_t)kRtLaneWarps * 32 * 16 * (a.E / 8 | 1);
  return cudaLaunchKernelEx(&cfg, kern, a, csize, FastDiv((uint32_t)(a.E / 8)));
}

size_t router_ws_bytes(int T, int E) {
  const int n = router_grid(T).clusters;
  return n > 1 ? (size_t)n * ((size_t)E * 8 + 8) : 0;
}

tm_status router_check(const char* what, const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t E,
                       int32_t k) {
  if (!dtype_ok(dtype)) return status_fail(TM_EINVAL, "%s: dtype=%d is not a tm_dtype", what, dtype);
  if (T < 0) return status_fail(TM_EINVAL, "%s: T=%d < 0", what, T);
  if (T > 1 << 30) return status_fail(TM_EUNSUPPORTED, "%s: T=%d is more than %d", what, T, 1 << 30);
  if (E < 1 || E > kMaxExperts) return status_fail(TM_EUNSUPPORTED, "%s: E=%d outside 1..%d", what, E, kMaxExperts);
  if (k < 1 || k > 32 || k > E) return status_fail(TM_EINVAL, "%s: k=%d outside 1..min(E,32)", what, k);
  if (ld < E) return status_fail(TM_EINVAL, "%s: ld=%lld is less than E=%d", what, (long long)ld, E);
  if (T > 0 && !logits) return status_fail(TM_EINVAL, "%s: logits is NULL", what);
  if (((uintptr_t)logits) % dtype_bytes(dtype))
    return status_fail(TM_EINVAL, "%s: logits must be aligned to its elements", what);
  return TM_OK;
}

}  // namespace

}  // namespace tmoe

using namespace tmoe;

extern "C" {

size_t trellis_moe_router_workspace_size(int32_t T, int32_t E) {
  if (T < 0 || T > 1 << 30 || E < 1 || E > kMaxExperts) return 0;
  return router_ws_bytes(T, E);
}

tm_status trellis_moe_router_forward(const void* logits, int32_t dtype, int64_t ld, const uint8_t* mask, int32_t T,
                                     int32_t E, int32_t k, int32_t* ids, float* w, float* lse, int32_t* counts,
                                     float* prob, float* losses, int32_t* tokens, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  set_last_error("");
  const tm_status s = router_check("router", logits, dtype, ld, T, E, k);
  if (s != TM_OK) return s;
  if (!counts || !prob || !losses || !tokens)
    return status_fail(TM_EINVAL, "counts, prob, losses and tokens must be non-NULL");
  if (T > 0 && (!ids || !w || !lse)) return status_fail(TM_EINVAL, "ids, w and lse must be non-NULL");
  const size_t need = router_ws_bytes(T, E);
  if (need > 0) {
    if (!workspace) return status_fail(TM_EWORKSPACE, "workspace is NULL");
    if (((uintptr_t)workspace) % 16) return status_fail(TM_EWORKSPACE, "workspace must be 16-byte aligned");
    if (workspace_bytes < need)
      return status_fail(TM_EWORKSPACE, "workspace has %zu bytes, %zu needed for T=%d E=%d", workspace_bytes, need, T, E);
  }
  cudaStream_t st = (cudaStream_t)stream;
  RouterFwd a{logits, ld, mask, T, E, k, ids, w, lse, counts, prob, losses, tokens, nullptr, nullptr, nullptr, nullptr};
  const bool lanes = router_lanes(a, dtype);
  const int csize = router_grid(T).csize;
  int clusters = router_grid(T).clusters;
  // (32 tokens a warp, spread over the CTAs; rows of more than 208 experts leave room for one CTA an SM)
  if (lanes) clusters = std::min(std::min(clusters, E > 208 ? kRtMaxClusters / 2 : kRtMaxClusters), ((T + 31) / 32 + 1) / 2);
  a.part_prob = static_cast<float*>(workspace);
  a.part_counts = reinterpret_cast<int32_t*>(a.part_prob + (size_t)clusters * E);
  a.part_z = reinterpret_cast<float*>(a.part_counts + (size_t)clusters * E);
  a.part_n = reinterpret_cast<int32_t*>(a.part_z + clusters);
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(clusters * csize));
  cfg.blockDim = dim3(32 * kRtWarps);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = csize > 1 ? 2 : 1;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {(unsigned)csize, 1, 1};
  cudaError_t e = by_pairs(dtype, E, logits, ld, nullptr, [&](auto elem, auto pair) {
    using T16 = std::conditional_t<std::is_same<decltype(elem), __half>::value, __half, __nv_bfloat16>;
    return by_width(E, [&](auto v) {
      if (lanes) return router_lanes_launch<decltype(v)::value, T16>(a, cfg, csize);
      return cudaLaunchKernelEx(&cfg, k_router_fwd<decltype(v)::value, decltype(elem), decltype(pair)::value>, a, csize);
    });
  });
  if (e == cudaSuccess && clusters > 1) {
    e = launch_after(k_router_finish, dim3(kFinCtas), kMaxExperts, 0, st, a, clusters);
  }
  return e == cudaSuccess ? TM_OK : status_cuda(e, "router with losses");
}

tm_status trellis_moe_router_backward(const void* logits, int32_t dtype, int64_t ld, const uint8_t* mask, int32_t T,
                                      int32_t E, int32_t k, const int32_t* ids, const float* w, const float* lse,
                                      const int32_t* counts, const int32_t* tokens, const float* grad_w,
                                      const float* grad_losses, void* grad_logits, void* stream) {
  set_last_error("");
  const tm_status s = router_check("router backward", logits, dtype, ld, T, E, k);
  if (s != TM_OK) return s;
  if (T == 0) return TM_OK;
  if (!lse || !counts || !tokens || !grad_logits)
    return status_fail(TM_EINVAL, "lse, counts, tokens and grad_logits must be non-NULL");
  if (grad_w && (!ids || !w)) return status_fail(TM_EINVAL, "ids and w must be non-NULL with grad_w");
  if (((uintptr_t)grad_logits) % dtype_bytes(dtype))
    return status_fail(TM_EINVAL, "grad_logits must be aligned to its elements");
  RouterBwd a{logits, ld, mask, T, E, k, ids, w, lse, counts, tokens, grad_w, grad_losses, grad_logits};
  cudaStream_t st = (cudaStream_t)stream;
  const int ctas = std::min(152 * kRtBwdCtas, (T + 7) / 8);
  const cudaError_t e = by_pairs(dtype, E, logits, ld, grad_logits, [&](auto elem, auto pair) {
    return by_width(E, [&](auto v) {
      return launch_after(k_router_bwd<decltype(v)::value, decltype(elem), decltype(pair)::value>, dim3(ctas), 256, 0, st, a);
    });
  });
  return e == cudaSuccess ? TM_OK : status_cuda(e, "router backward");
}

}  // extern "C"
