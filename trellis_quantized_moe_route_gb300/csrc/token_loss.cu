// Log probabilities of given tokens, and distillation from a teacher's largest
// logits (sm_103a). With u = l / tau, m = max l, s = ln sum exp((l - m) / tau):
//   log p_i = (l_i - m) / tau - s,   H = s - sum p_i (l_i - m) / tau
//   dl_i    = (g ([i = y] - p_i) - h p_i (log p_i + H)) / tau
//   loss    = sum_j q_j (ln q_j - log p_(i_j)),   dl_i = g (Q p_i - sum_(j: i_j = i) q_j) / tau
// One CTA a row; the simplest form.
#include <algorithm>
#include <cmath>

#include "elem.cuh"
#include "pdl.cuh"
#include "status.h"

namespace tmoe {

namespace {

constexpr int kTlThreads = 512;
constexpr int kTlMaxTop = 32;
constexpr int kTlMaxEntries = 256;
constexpr float kLog2e = 1.4426950408889634f;

struct TlArgs {
  const void* logits;
  int64_t ld;
  int T, V;
  float inv_tau;
  // given tokens
  const void* targets;
  int target64, top;
  float *logprob, *entropy, *stats, *top_logprobs;
  int32_t* top_ids;
  const float *grad_logprob, *grad_entropy;
  // teacher
  const void* ids;
  const void* values;
  int ids64, values_dtype, n;
  const uint8_t* mask;
  const float* teacher_lse;
  float* loss;
  const float* grad_loss;
  void* grad;
  int64_t grad_ld;
};

// Values as whole numbers in their order, NaN (of either sign) above all, -0 as 0.
__device__ __forceinline__ uint32_t tl_order(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ long tl_index(const void* p, int is64, size_t i) {
  return is64 ? (long)static_cast<const int64_t*>(p)[i] : (long)static_cast<const int32_t*>(p)[i];
}

template <typename V, typename F>
__device__ __forceinline__ V tl_reduce(V v, F f, V* s) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s[0];
  for (int w = 1; w < kTlThreads / 32; ++w) v = f(v, s[w]);
  return v;
}

__device__ __forceinline__ float tl_max_nan(float a, float b) { return a != a ? a : (b != b ? b : fmaxf(a, b)); }

// m (0 where the row is -inf throughout) and s of a row, and sum p u'
template <typename T>
__device__ void tl_stats(const T* row, int V, float inv_tau, float& m, float& s, float& pu, float* sh) {
  float mx = -INFINITY;
  for (int i = threadIdx.x; i < V; i += kTlThreads) mx = tl_max_nan(mx, to_f32(row[i]));
  mx = tl_reduce(mx, tl_max_nan, sh);
  m = mx == -INFINITY ? 0.0f : mx;
  float sum = 0, dot = 0;
  for (int i = threadIdx.x; i < V; i += kTlThreads) {
    const float u = fmaxf((to_f32(row[i]) - m) * inv_tau, -1000.0f), e = expf(u);
    sum += e;
    dot += e * u;
  }
  auto add = [](float a, float b) { return a + b; };
  sum = tl_reduce(sum, add, sh);
  dot = tl_reduce(dot, add, sh);
  s = mx != mx || mx == INFINITY ? NAN : logf(sum);
  pu = mx == -INFINITY ? 0.0f : dot / sum;
  if (mx == -INFINITY) s = -INFINITY;
}

template <typename T>
__global__ void __launch_bounds__(kTlThreads) k_token_logprobs(const TlArgs a) {
  __shared__ float sh[32];
  __shared__ unsigned long long shk[32];
  for (long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    float m, s, pu;
    tl_stats(row, a.V, a.inv_tau, m, s, pu, sh);
    const bool none = s == -INFINITY;
    if (threadIdx.x == 0) {
      const long y = tl_index(a.targets, a.target64, t);
      a.logprob[t] = y < 0 || y >= a.V ? 0.0f : none ? -INFINITY : (to_f32(row[y]) - m) * a.inv_tau - s;
      a.entropy[t] = none ? 0.0f : s - pu;
      a.stats[2 * t] = m;
      a.stats[2 * t + 1] = s;
    }
    unsigned long long last = ~0ull;
    for (int j = 0; j < a.top; ++j) {
      unsigned long long best = 0;
      for (int i = threadIdx.x; i < a.V; i += kTlThreads) {
        const unsigned long long k = ((unsigned long long)tl_order(to_f32(row[i])) << 32) | (uint32_t)~i;
        if ((j == 0 || k < last) && k > best) best = k;
      }
      best = tl_reduce(best, [](unsigned long long x, unsigned long long y) { return x > y ? x : y; }, shk);
      last = best;
      if (threadIdx.x == 0) {
        const int i = (int)~(uint32_t)best;
        a.top_ids[t * a.top + j] = i;
        a.top_logprobs[t * a.top + j] = none ? -INFINITY : (to_f32(row[i]) - m) * a.inv_tau - s;
      }
    }
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(kTlThreads) k_token_logprobs_bwd(const TlArgs a) {
  for (long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    T* out = static_cast<T*>(a.grad) + t * a.grad_ld;
    const long y = tl_index(a.targets, a.target64, t);
    const float m = a.stats[2 * t], s = a.stats[2 * t + 1], H = a.entropy[t];
    const float g = y < 0 || y >= a.V || !a.grad_logprob ? 0.0f : a.grad_logprob[t], h = a.grad_entropy ? a.grad_entropy[t] : 0.0f;
    for (int i = threadIdx.x; i < a.V; i += kTlThreads) {
      const float lp = s == -INFINITY ? -1000.0f : fmaxf((to_f32(row[i]) - m) * a.inv_tau, -1000.0f) - s;
      const float p = expf(lp);
      out[i] = from_f32<T>((g * ((i == y ? 1.0f : 0.0f) - p) - h * p * (lp + H)) * a.inv_tau);
    }
  }
}

// The teacher's entries of a row in shared memory: id (-1: none), q, ln q; returns Q.
struct TlTeacher {
  int id[kTlMaxEntries];
  float q[kTlMaxEntries], lnq[kTlMaxEntries], logit[kTlMaxEntries];
};

__device__ __forceinline__ float tl_value(const TlArgs& a, size_t i) {
  return a.values_dtype == TM_F32    ? static_cast<const float*>(a.values)[i]
         : a.values_dtype == TM_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(a.values)[i])
                                     : to_f32(static_cast<const __half*>(a.values)[i]);
}

template <typename T>
__device__ float tl_teacher(const TlArgs& a, long t, const T* row, TlTeacher& te, float* sh) {
  const int j = threadIdx.x;
  float v = -INFINITY;
  if (j < a.n) {
    const long id = tl_index(a.ids, a.ids64, t * a.n + j);
    te.id[j] = id < 0 || id >= a.V ? -1 : (int)id;
    if (te.id[j] >= 0) {
      v = tl_value(a, t * a.n + j);
      te.logit[j] = to_f32(row[te.id[j]]);
    }
  }
  auto add = [](float x, float y) { return x + y; };
  float lnq;
  if (a.teacher_lse) {
    lnq = v * a.inv_tau - a.teacher_lse[t];
    if (v == -INFINITY) lnq = v;
  } else {
    float m = tl_reduce(v, tl_max_nan, sh);
    if (m == -INFINITY) m = 0.0f;
    const float u = (v - m) * a.inv_tau;
    lnq = u - logf(tl_reduce(expf(u), add, sh));
    if (v == -INFINITY) lnq = v;
  }
  const float q = expf(lnq);
  if (j < a.n) {
    te.q[j] = q;
    te.lnq[j] = lnq;
  }
  return tl_reduce(q, add, sh);
}

// STATS: from the row (else read back); LOSS, GRAD: what is written.
template <typename T, bool FWD, bool GRAD>
__global__ void __launch_bounds__(kTlThreads) k_distill(const TlArgs a) {
  __shared__ float sh[32];
  __shared__ TlTeacher te;
  auto add = [](float x, float y) { return x + y; };
  for (long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    T* out = static_cast<T*>(a.grad) + t * a.grad_ld;
    if (a.mask && !a.mask[t]) {
      if (GRAD)
        for (int i = threadIdx.x; i < a.V; i += kTlThreads) out[i] = from_f32<T>(0.0f);
      if (FWD && threadIdx.x == 0) {
        a.loss[t] = 0.0f;
        if (a.stats) a.stats[2 * t] = a.stats[2 * t + 1] = 0.0f;
      }
      continue;
    }
    const float Q = tl_teacher(a, t, row, te, sh);
    float m, s, pu;
    if (FWD) {
      tl_stats(row, a.V, a.inv_tau, m, s, pu, sh);
      const int j = threadIdx.x;
      float term = 0.0f;
      if (j < a.n && te.id[j] >= 0 && !(te.q[j] == 0.0f)) {
        const float lp = s == -INFINITY ? -INFINITY : (te.logit[j] - m) * a.inv_tau - s;
        term = te.q[j] * (te.lnq[j] - lp);
      }
      term = tl_reduce(term, add, sh);
      if (threadIdx.x == 0) {
        a.loss[t] = term;
        if (a.stats) {
          a.stats[2 * t] = m;
          a.stats[2 * t + 1] = s;
        }
      }
    } else {
      m = a.stats[2 * t], s = a.stats[2 * t + 1];
    }
    __syncthreads();
    if (GRAD) {
      const float g = a.grad_loss[t] * a.inv_tau;
      auto prob = [&](float l) { return s == -INFINITY ? 0.0f : expf(fmaxf((l - m) * a.inv_tau, -1000.0f) - s); };
      for (int i = threadIdx.x; i < a.V; i += kTlThreads) out[i] = from_f32<T>(g * Q * prob(to_f32(row[i])));
      __syncthreads();
      const int j = threadIdx.x;
      if (j < a.n && te.id[j] >= 0) {
        bool first = true;
        float q = 0.0f;
        for (int x = 0; x < a.n; ++x)
          if (te.id[x] == te.id[j]) {
            if (x < j) first = false;
            q += te.q[x];
          }
        if (first) out[te.id[j]] = from_f32<T>(g * (Q * prob(te.logit[j]) - q));
      }
    }
    __syncthreads();
  }
}

int tl_ctas(int T) { return std::min(T, 152 * 4); }

tm_status tl_check(const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t V, float temperature) {
  if (!dtype_ok(dtype)) return status_fail(TM_EINVAL, "dtype=%d is not a tm_dtype", dtype);
  if (T < 0) return status_fail(TM_EINVAL, "T=%d < 0", T);
  if (V < 1 || V > (1 << 30)) return status_fail(TM_EINVAL, "V=%d outside 1..%d", V, 1 << 30);
  if (ld < V) return status_fail(TM_EINVAL, "ld=%lld is less than V=%d", (long long)ld, V);
  if (!(temperature > 0.0f) || std::isinf(temperature) || std::isinf(kLog2e / temperature))
    return status_fail(TM_EINVAL, "temperature=%g is not a positive number whose reciprocal is one", temperature);
  if (T > 0 && !logits) return status_fail(TM_EINVAL, "logits must be non-NULL");
  if (((uintptr_t)logits) % dtype_bytes(dtype)) return status_fail(TM_EINVAL, "logits must be aligned to its elements");
  return TM_OK;
}

tm_status tl_check_grad(const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t V, const void* grad, int64_t grad_ld) {
  if (grad_ld < V) return status_fail(TM_EINVAL, "grad_ld=%lld is less than V=%d", (long long)grad_ld, V);
  if (T > 0 && !grad) return status_fail(TM_EINVAL, "grad_logits must be non-NULL");
  if (((uintptr_t)grad) % dtype_bytes(dtype)) return status_fail(TM_EINVAL, "grad_logits must be aligned to its elements");
  if (T > 0 && !(grad == logits && grad_ld == ld)) {
    const uintptr_t es = dtype_bytes(dtype), a0 = (uintptr_t)logits, b0 = (uintptr_t)grad;
    const uintptr_t a1 = a0 + ((uintptr_t)(T - 1) * ld + V) * es, b1 = b0 + ((uintptr_t)(T - 1) * grad_ld + V) * es;
    // (rows of one buffer may lie between those of the other: a column range of the same tensor)
    const uintptr_t step = (uintptr_t)ld * es, off = b0 > a0 ? (b0 - a0) % step : step - 1 - (a0 - b0 - 1) % step;
    const bool beside = ld == grad_ld && off >= V * es && step - off >= V * es;
    if (a0 < b1 && b0 < a1 && !beside)
      return status_fail(TM_EINVAL, "grad_logits must be logits itself, with the same row stride, or lie apart from it");
  }
  return TM_OK;
}

tm_status tl_check_teacher(const TlArgs& a, int32_t id_bytes, int32_t n) {
  if (id_bytes != 4 && id_bytes != 8) return status_fail(TM_EINVAL, "id_bytes=%d: ids have 4 or 8 bytes", id_bytes);
  if (!dtype_ok(a.values_dtype)) return status_fail(TM_EINVAL, "values_dtype=%d is not a tm_dtype", a.values_dtype);
  if (n < 1 || n > kTlMaxEntries) return status_fail(TM_EINVAL, "n=%d outside 1..%d", n, kTlMaxEntries);
  if (a.T > 0 && (!a.ids || !a.values)) return status_fail(TM_EINVAL, "ids and values must be non-NULL");
  return TM_OK;
}

template <bool FWD, bool GRAD>
tm_status tl_distill(const TlArgs& a, int32_t dtype, void* stream) {
  if (a.T == 0) return TM_OK;
  auto go = [&](auto elem) {
    k_distill<decltype(elem), FWD, GRAD><<<tl_ctas(a.T), kTlThreads, 0, (cudaStream_t)stream>>>(a);
    return cudaGetLastError();
  };
  const cudaError_t e = TM_BY_DTYPE(dtype, go);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "distillation");
}

TlArgs tl_teacher_args(const void* logits, int64_t ld, const void* ids, int32_t id_bytes, const void* values,
                       int32_t values_dtype, int32_t n, const uint8_t* mask, const float* teacher_lse, int32_t T, int32_t V,
                       float temperature) {
  TlArgs a{};
  a.logits = logits, a.ld = ld, a.T = T, a.V = V, a.inv_tau = 1.0f / temperature;
  a.ids = ids, a.ids64 = id_bytes == 8, a.values = values, a.values_dtype = values_dtype, a.n = n;
  a.mask = mask, a.teacher_lse = teacher_lse;
  return a;
}

}  // namespace

}  // namespace tmoe

using namespace tmoe;

extern "C" {

tm_status trellis_moe_token_logprobs(const void* logits, int32_t dtype, int64_t ld, const void* targets,
                                     int32_t target_bytes, int32_t T, int32_t V, float temperature, int32_t top,
                                     float* logprob, float* entropy, float* stats, int32_t* top_ids, float* top_logprobs,
                                     void* stream) {
  set_last_error("");
  tm_status st = tl_check(logits, dtype, ld, T, V, temperature);
  if (st != TM_OK) return st;
  if (target_bytes != 4 && target_bytes != 8)
    return status_fail(TM_EINVAL, "target_bytes=%d: targets have 4 or 8 bytes", target_bytes);
  if (top < 0 || top > kTlMaxTop || top > V) return status_fail(TM_EINVAL, "top=%d outside 0..min(V,%d)", top, kTlMaxTop);
  if (T == 0) return TM_OK;
  if (!targets || !logprob || !entropy || !stats) return status_fail(TM_EINVAL, "targets, logprob, entropy and stats must be non-NULL");
  if (top > 0 && (!top_ids || !top_logprobs)) return status_fail(TM_EINVAL, "top_ids and top_logprobs must be non-NULL");
  TlArgs a{};
  a.logits = logits, a.ld = ld, a.T = T, a.V = V, a.inv_tau = 1.0f / temperature;
  a.targets = targets, a.target64 = target_bytes == 8, a.top = top;
  a.logprob = logprob, a.entropy = entropy, a.stats = stats, a.top_ids = top_ids, a.top_logprobs = top_logprobs;
  auto go = [&](auto elem) {
    k_token_logprobs<decltype(elem)><<<tl_ctas(T), kTlThreads, 0, (cudaStream_t)stream>>>(a);
    return cudaGetLastError();
  };
  const cudaError_t e = TM_BY_DTYPE(dtype, go);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "token log probabilities");
}

tm_status trellis_moe_token_logprobs_backward(const void* logits, int32_t dtype, int64_t ld, const void* targets,
                                              int32_t target_bytes, int32_t T, int32_t V, float temperature,
                                              const float* entropy, const float* stats, const float* grad_logprob,
                                              const float* grad_entropy, void* grad_logits, int64_t grad_ld, void* stream) {
  set_last_error("");
  tm_status st = tl_check(logits, dtype, ld, T, V, temperature);
  if (st == TM_OK) st = tl_check_grad(logits, dtype, ld, T, V, grad_logits, grad_ld);
  if (st != TM_OK) return st;
  if (target_bytes != 4 && target_bytes != 8)
    return status_fail(TM_EINVAL, "target_bytes=%d: targets have 4 or 8 bytes", target_bytes);
  if (T == 0) return TM_OK;
  if (!targets || !entropy || !stats) return status_fail(TM_EINVAL, "targets, entropy and stats must be non-NULL");
  TlArgs a{};
  a.logits = logits, a.ld = ld, a.T = T, a.V = V, a.inv_tau = 1.0f / temperature;
  a.targets = targets, a.target64 = target_bytes == 8;
  a.entropy = const_cast<float*>(entropy), a.stats = const_cast<float*>(stats);
  a.grad_logprob = grad_logprob, a.grad_entropy = grad_entropy, a.grad = grad_logits, a.grad_ld = grad_ld;
  auto go = [&](auto elem) {
    k_token_logprobs_bwd<decltype(elem)><<<tl_ctas(T), kTlThreads, 0, (cudaStream_t)stream>>>(a);
    return cudaGetLastError();
  };
  const cudaError_t e = TM_BY_DTYPE(dtype, go);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "token log probabilities backward");
}

tm_status trellis_moe_distill_forward(const void* logits, int32_t dtype, int64_t ld, const void* ids, int32_t id_bytes,
                                      const void* values, int32_t values_dtype, int32_t n, const uint8_t* mask,
                                      const float* teacher_lse, int32_t T, int32_t V, float temperature, float* loss,
                                      float* stats, void* stream) {
  set_last_error("");
  TlArgs a = tl_teacher_args(logits, ld, ids, id_bytes, values, values_dtype, n, mask, teacher_lse, T, V, temperature);
  tm_status st = tl_check(logits, dtype, ld, T, V, temperature);
  if (st == TM_OK) st = tl_check_teacher(a, id_bytes, n);
  if (st != TM_OK) return st;
  if (T > 0 && (!loss || !stats)) return status_fail(TM_EINVAL, "loss and stats must be non-NULL");
  a.loss = loss, a.stats = stats;
  return tl_distill<true, false>(a, dtype, stream);
}

tm_status trellis_moe_distill_backward(const void* logits, int32_t dtype, int64_t ld, const void* ids, int32_t id_bytes,
                                       const void* values, int32_t values_dtype, int32_t n, const uint8_t* mask,
                                       const float* teacher_lse, int32_t T, int32_t V, float temperature,
                                       const float* stats, const float* grad_loss, void* grad_logits, int64_t grad_ld,
                                       void* stream) {
  set_last_error("");
  TlArgs a = tl_teacher_args(logits, ld, ids, id_bytes, values, values_dtype, n, mask, teacher_lse, T, V, temperature);
  tm_status st = tl_check(logits, dtype, ld, T, V, temperature);
  if (st == TM_OK) st = tl_check_teacher(a, id_bytes, n);
  if (st == TM_OK) st = tl_check_grad(logits, dtype, ld, T, V, grad_logits, grad_ld);
  if (st != TM_OK) return st;
  if (T > 0 && (!grad_loss || !stats)) return status_fail(TM_EINVAL, "stats and grad_loss must be non-NULL");
  a.stats = const_cast<float*>(stats), a.grad_loss = grad_loss, a.grad = grad_logits, a.grad_ld = grad_ld;
  return tl_distill<false, true>(a, dtype, stream);
}

tm_status trellis_moe_distill_loss_grad(const void* logits, int32_t dtype, int64_t ld, const void* ids, int32_t id_bytes,
                                        const void* values, int32_t values_dtype, int32_t n, const uint8_t* mask,
                                        const float* teacher_lse, int32_t T, int32_t V, float temperature,
                                        const float* grad_loss, float* loss, void* grad_logits, int64_t grad_ld,
                                        void* stream) {
  set_last_error("");
  TlArgs a = tl_teacher_args(logits, ld, ids, id_bytes, values, values_dtype, n, mask, teacher_lse, T, V, temperature);
  tm_status st = tl_check(logits, dtype, ld, T, V, temperature);
  if (st == TM_OK) st = tl_check_teacher(a, id_bytes, n);
  if (st == TM_OK) st = tl_check_grad(logits, dtype, ld, T, V, grad_logits, grad_ld);
  if (st != TM_OK) return st;
  if (T > 0 && (!grad_loss || !loss)) return status_fail(TM_EINVAL, "grad_loss and loss must be non-NULL");
  a.loss = loss, a.grad_loss = grad_loss, a.grad = grad_logits, a.grad_ld = grad_ld;
  return tl_distill<true, true>(a, dtype, stream);
}

}  // extern "C"
