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
// One warp takes a token: expert e = lane + 32 i sits in register i of its
// lane, so a row is read once, coalesced, with no alignment asked for. The
// statistics stay in registers over all of a warp's tokens, are added over the
// CTA's warps in shared memory and over the CTAs by a second kernel, always in
// the same order: no atomics, the same bits every time. The backward pass
// reads the logits again and rebuilds p from lse, which costs less than
// storing p (T E fp32).
#include <algorithm>

#include "elem.cuh"
#include "status.h"

namespace tmoe {

namespace {

constexpr int kRtWarps = 16;      // warps of a CTA with many tokens
constexpr int kRtMaxCtas = 304;   // two CTAs of 512 threads on each of 152 SMs

__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);  // -0 as +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float order_unkey(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

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
  // per CTA: [E] probability sums, [E] counts, then sum lse^2 and valid tokens
  float* part_prob;
  int32_t* part_counts;
  float* part_z;
  int32_t* part_n;
};

// Adds up `parts` CTAs' statistics and writes the results: a warp adds every
// (warps)-th part in order, then one thread an expert adds the warps' sums.
template <int V>
__device__ void router_finish(const RouterFwd& a, int parts, float (*s_acc)[V * 32], int (*s_cnt)[V * 32]) {
  __shared__ float s_dot[32];
  __shared__ int s_n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  float acc[V] = {};
  int cnt[V] = {};
  for (int c0 = warp; c0 < parts; c0 += warps * 4) {
    float p[4][V];
    int n[4][V];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = c0 + u * warps, e = lane + 32 * i;
        const bool in = c < parts && e < a.E;
        p[u][i] = in ? a.part_prob[(size_t)c * a.E + e] : 0.0f;
        n[u][i] = in ? a.part_counts[(size_t)c * a.E + e] : 0;
      }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        acc[i] += p[u][i];
        cnt[i] += n[u][i];
      }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    s_acc[warp][lane + 32 * i] = acc[i];
    s_cnt[warp][lane + 32 * i] = cnt[i];
  }
  if (warp == 0) {
    int n = 0;
    float z = 0.0f;
    for (int c = lane; c < parts; c += 32) {
      n += a.part_n[c];
      z += a.part_z[c];
    }
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    z = warp_sum(z);
    if (lane == 0) {
      s_n = n;
      *a.tokens = n;
      a.losses[1] = n > 0 ? z / (float)n : 0.0f;
    }
  }
  __syncthreads();
  const float inv_n = s_n > 0 ? 1.0f / (float)s_n : 0.0f;
  float dot = 0.0f;
  if (tid < a.E) {
    float p = 0.0f;
    int c = 0;
    for (int u = 0; u < warps; ++u) {
      p += s_acc[u][tid];
      c += s_cnt[u][tid];
    }
    p *= inv_n;
    a.prob[tid] = p;
    a.counts[tid] = c;
    dot = (float)c * inv_n / (float)a.k * p;
  }
  dot = warp_sum(dot);
  if (lane == 0) s_dot[warp] = dot;
  __syncthreads();
  if (warp == 0) {
    dot = lane < warps ? s_dot[lane] : 0.0f;
    dot = warp_sum(dot);
    if (lane == 0) a.losses[0] = (float)a.E * dot;
  }
}

// Keys of one token, expert lane + 32 i in place i (absent: 0, below every
// float's), sorted descending within the lane; `perm` holds the places they
// came from, four bits each, equal keys in order of place.
template <int V>
__device__ __forceinline__ void router_sort(uint32_t (&key)[V], uint32_t& perm) {
  uint32_t id[V];
#pragma unroll
  for (int i = 0; i < V; ++i) id[i] = i;
  // odd-even transposition: neighbours swap only when out of order, so it is stable
#pragma unroll
  for (int r = 0; r < V; ++r)
#pragma unroll
    for (int i = r & 1; i + 1 < V; i += 2) {
      const bool sw = key[i + 1] > key[i];
      const uint32_t k0 = key[i], k1 = key[i + 1], d0 = id[i], d1 = id[i + 1];
      key[i] = sw ? k1 : k0;
      key[i + 1] = sw ? k0 : k1;
      id[i] = sw ? d1 : d0;
      id[i + 1] = sw ? d0 : d1;
    }
  perm = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) perm |= id[i] << (4 * i);
}

// One token by one warp: l[i] is the logit of expert lane + 32 i. The k rounds
// take the largest of the lanes' first keys; the lane it came from moves its
// keys up by one. Adds the token's statistics to the lane's sums.
template <int V>
__device__ __forceinline__ void router_token(const RouterFwd& a, int t, const float (&l)[V], bool on,
                                             float (&acc)[V], int (&cnt)[V], float& z, int& n) {
  const int lane = threadIdx.x & 31;
  uint32_t key[V], perm;
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = lane + 32 * i < a.E ? order_key(l[i]) : 0u;
  router_sort<V>(key, perm);
  uint32_t sel = 0;  // bit i: expert lane + 32 i was selected
  uint32_t my_key = 0, my_id = 0, first = 0;
  for (int j = 0; j < a.k; ++j) {
    const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, key[0]);
    const uint32_t id = lane + 32 * (perm & 15u);
    uint32_t who = __ballot_sync(0xFFFFFFFFu, key[0] == best);
    uint32_t winner = __ffs(who) - 1;
    uint32_t wid = __shfl_sync(0xFFFFFFFFu, id, winner);
    if (who & (who - 1)) {  // equal logits: the lowest expert
      wid = __reduce_min_sync(0xFFFFFFFFu, key[0] == best ? id : 0xFFFFFFFFu);
      winner = wid & 31u;
    }
    if (j == 0) first = best;
    if (lane == j) {
      my_key = best;
      my_id = wid;
    }
    if (lane == (int)winner) {
      sel |= 1u << (perm & 15u);
      perm >>= 4;
#pragma unroll
      for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
      key[V - 1] = 0u;
    }
  }
  const float m = order_unkey(first);
  const bool some = m != -INFINITY;
  float p[V], total = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    p[i] = lane + 32 * i < a.E ? __expf(l[i] - m) : 0.0f;
    total += p[i];
  }
  total = warp_sum(total);
  const float we = lane < a.k ? __expf(order_unkey(my_key) - m) : 0.0f;
  const float wsum = warp_sum(we);
  const float lse = m + logf(total);
  if (lane < a.k) {
    a.ids[(size_t)t * a.k + lane] = (int)my_id;
    a.w[(size_t)t * a.k + lane] = some ? we / wsum : 0.0f;
  }
  if (lane == 0) a.lse[t] = some ? lse : -INFINITY;
  if (on && some) {
    const float inv = 1.0f / total;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      acc[i] += p[i] * inv;
      if ((sel >> i & 1u) && l[i] != -INFINITY) ++cnt[i];
    }
    z += lse * lse;
    ++n;
  }
}

// A warp's tokens are warp, warp + W, ... (W: warps of the grid). With one CTA
// the statistics are finished here.
template <int V, typename T>
__global__ void __launch_bounds__(kRtWarps * 32) k_router_fwd(RouterFwd a) {
  __shared__ float s_acc[kRtWarps][V * 32];
  __shared__ int s_cnt[kRtWarps][V * 32];
  __shared__ float s_z[kRtWarps];
  __shared__ int s_nv[kRtWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const T* logits = static_cast<const T*>(a.logits);
  float acc[V] = {};
  int cnt[V] = {};
  float z = 0.0f;
  int n = 0;
  for (int t = blockIdx.x * warps + warp; t < a.T; t += gridDim.x * warps) {
    const T* row = logits + (size_t)t * a.ld;
    float l[V];
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = lane + 32 * i < a.E ? to_f32(row[lane + 32 * i]) : 0.0f;
    router_token<V>(a, t, l, a.mask == nullptr || a.mask[t] != 0, acc, cnt, z, n);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    s_acc[warp][lane + 32 * i] = acc[i];
    s_cnt[warp][lane + 32 * i] = cnt[i];
  }
  if (lane == 0) {
    s_z[warp] = z;
    s_nv[warp] = n;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    float p = 0.0f;
    int c = 0;
    for (int u = 0; u < warps; ++u) {
      p += s_acc[u][e];
      c += s_cnt[u][e];
    }
    a.part_prob[(size_t)blockIdx.x * a.E + e] = p;
    a.part_counts[(size_t)blockIdx.x * a.E + e] = c;
  }
  if (threadIdx.x == 0) {
    float zs = 0.0f;
    int ns = 0;
    for (int u = 0; u < warps; ++u) {
      zs += s_z[u];
      ns += s_nv[u];
    }
    a.part_z[blockIdx.x] = zs;
    a.part_n[blockIdx.x] = ns;
  }
  if (gridDim.x == 1) {
    __syncthreads();
    router_finish<V>(a, 1, s_acc, s_cnt);
  }
}

template <int V>
__global__ void __launch_bounds__(kRtWarps * 32) k_router_finish(RouterFwd a, int parts) {
  __shared__ float s_acc[kRtWarps][V * 32];
  __shared__ int s_cnt[kRtWarps][V * 32];
  router_finish<V>(a, parts, s_acc, s_cnt);
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

template <int V, typename T>
__global__ void __launch_bounds__(256) k_router_bwd(RouterBwd a) {
  __shared__ float s_sel[8][V * 32];  // each warp's selected experts' gradients, zero between tokens
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* logits = static_cast<const T*>(a.logits);
  T* grad = static_cast<T*>(a.grad_logits);
  const int n = *a.tokens;
  const float inv_n = n > 0 ? 1.0f / (float)n : 0.0f;
  const float gb = a.grad_losses ? a.grad_losses[0] * (float)a.E * inv_n : 0.0f;
  const float gz = a.grad_losses ? a.grad_losses[1] * 2.0f * inv_n : 0.0f;
  float f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    f[i] = lane + 32 * i < a.E ? (float)a.counts[lane + 32 * i] * inv_n / (float)a.k : 0.0f;
    s_sel[warp][lane + 32 * i] = 0.0f;
  }
  __syncwarp();
  for (int t = blockIdx.x * 8 + warp; t < a.T; t += gridDim.x * 8) {
    const T* row = logits + (size_t)t * a.ld;
    const float lse = a.lse[t];
    const bool on = lse != -INFINITY && (a.mask == nullptr || a.mask[t] != 0);
    float p[V], s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = on && lane + 32 * i < a.E ? __expf(to_f32(row[lane + 32 * i]) - lse) : 0.0f;
      s += f[i] * p[i];
    }
    s = warp_sum(s);
    int id = -1;
    if (a.grad_w) {
      float w = 0.0f, g = 0.0f;
      if (lane < a.k) {
        id = a.ids[(size_t)t * a.k + lane];
        w = a.w[(size_t)t * a.k + lane];
        g = a.grad_w[(size_t)t * a.k + lane];
      }
      // (a weight of zero gets no gradient whatever comes from above, and a
      // zero from above gives none whatever the weight: padding may hold NaN)
      const float wg = w != 0.0f && g != 0.0f ? w * g : 0.0f;
      const float dot = warp_sum(wg);
      if (id < 0 || id >= a.E) id = -1;
      if (id >= 0) s_sel[warp][id] = w != 0.0f && dot != 0.0f ? wg - w * dot : wg;
      __syncwarp();
    }
    const float c = gz * (on ? lse : 0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E) grad[(size_t)t * a.E + e] = from_f32<T>(p[i] * (gb * (f[i] - s) + c) + s_sel[warp][e]);
    }
    if (a.grad_w) {
      __syncwarp();
      if (id >= 0) s_sel[warp][id] = 0.0f;
      __syncwarp();
    }
  }
}

// Launches the instantiation of kernel K for E experts and element type T.
template <typename T, typename F>
cudaError_t by_width(int E, F f) {
  switch ((E + 31) / 32) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    case 7: return f(std::integral_constant<int, 7>());
    default: return f(std::integral_constant<int, 8>());
  }
}

int router_ctas(int T) { return std::min(kRtMaxCtas, (T + kRtWarps - 1) / kRtWarps); }

size_t router_ws_bytes(int T, int E) { return (size_t)std::max(1, router_ctas(T)) * ((size_t)E * 8 + 8); }

tm_status router_check(const char* what, const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t E,
                       int32_t k) {
  if (!dtype_ok(dtype)) return status_fail(TM_EINVAL, "%s: dtype=%d is not a tm_dtype", what, dtype);
  if (T < 0) return status_fail(TM_EINVAL, "%s: T=%d < 0", what, T);
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
  if (T < 0 || E < 1 || E > kMaxExperts) return 0;
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
  if (!workspace) return status_fail(TM_EWORKSPACE, "workspace is NULL");
  if (((uintptr_t)workspace) % 16) return status_fail(TM_EWORKSPACE, "workspace must be 16-byte aligned");
  if (workspace_bytes < need)
    return status_fail(TM_EWORKSPACE, "workspace has %zu bytes, %zu needed for T=%d E=%d", workspace_bytes, need, T, E);
  cudaStream_t st = (cudaStream_t)stream;
  RouterFwd a{logits, ld, mask, T, E, k, ids, w, lse, counts, prob, losses, tokens, nullptr, nullptr, nullptr, nullptr};
  const int ctas = std::max(1, router_ctas(T));
  a.part_prob = static_cast<float*>(workspace);
  a.part_counts = reinterpret_cast<int32_t*>(a.part_prob + (size_t)ctas * E);
  a.part_z = reinterpret_cast<float*>(a.part_counts + (size_t)ctas * E);
  a.part_n = reinterpret_cast<int32_t*>(a.part_z + ctas);
  const int threads = 32 * kRtWarps;
  auto go = [&](auto elem) {
    using T_ = decltype(elem);
    return by_width<T_>(E, [&](auto v) {
      constexpr int V = decltype(v)::value;
      k_router_fwd<V, T_><<<ctas, threads, 0, st>>>(a);
      if (ctas > 1) k_router_finish<V><<<1, threads, 0, st>>>(a, ctas);
      return cudaGetLastError();
    });
  };
  const cudaError_t e = TM_BY_DTYPE(dtype, go);
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
  const int ctas = std::min(152 * 8, (T + 7) / 8);
  auto go = [&](auto elem) {
    using T_ = decltype(elem);
    return by_width<T_>(E, [&](auto v) {
      k_router_bwd<decltype(v)::value, T_><<<ctas, 256, 0, st>>>(a);
      return cudaGetLastError();
    });
  };
  const cudaError_t e = TM_BY_DTYPE(dtype, go);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "router backward");
}

}  // extern "C"
