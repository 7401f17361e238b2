// Log probabilities of given tokens, and distillation from a teacher's largest
// logits (sm_103a). With u = l / tau, M = max l, s = ln sum exp((l - M) / tau):
//   log p_i = (l_i - M) / tau - s,   H = s - sum p_i (l_i - M) / tau
//   dl_i    = (g ([i = y] - p_i) - h p_i (log p_i + H)) / tau
//   loss    = sum_j q_j (ln q_j - log p_(i_j)),   dl_i = g (Q p_i - sum_(j: i_j = i) q_j) / tau
//
// Bound by memory: a row is read once (and its gradient written once). A row is
// cut into the segments of a cluster's CTAs; a CTA keeps its segment in shared
// memory, so that the pass that writes the gradient, and the search for the
// largest logits, need not read it again, and fetches the next row's while it
// works on this one (cp.async: a thread reads only words that it fetched itself,
// so that no barrier stands between). Longer rows go through in tiles.
#include <algorithm>
#include <cmath>

#include "elem.cuh"
#include "pdl.cuh"
#include "status.h"

namespace tmoe {

namespace {

constexpr int kTlMaxTop = 32;
constexpr int kTlMaxEntries = 256;
constexpr int kTlWords = 8;      // 16-byte words of a tile that a thread holds
constexpr int kTlCtas = 8;       // most CTAs of a cluster
constexpr int kTlCandidates = 448;  // (what lets three CTAs share an SM)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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
  int vec_out;           // the gradient's rows are aligned like the logits'
  int ctas, seg, tiles;  // CTAs of a row, words of a segment, tiles of a segment
};

// Values as whole numbers in their order, NaN (of either sign) above all, -0 as
// 0; 0 stands for no element.
__device__ __forceinline__ uint32_t tl_order(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float tl_value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ unsigned long long tl_key(uint32_t order, int i) {
  return ((unsigned long long)order << 32) | (uint32_t)~i;  // (of equal values the lower index is the larger key)
}

__device__ __forceinline__ long tl_index(const void* p, int is64, size_t i) {
  return is64 ? (long)static_cast<const int64_t*>(p)[i] : (long)static_cast<const int32_t*>(p)[i];
}

__device__ __forceinline__ float tl_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float tl_max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float tl_warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = tl_max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
__device__ __forceinline__ float tl_warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// 16 bytes of a row.
template <typename T>
struct TlWord {
  static constexpr int kN = 16 / (int)sizeof(T);
  uint4 q;
  __device__ __forceinline__ void to(float (&v)[kN]) const {
    const T* t = reinterpret_cast<const T*>(&q);
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = to_f32(t[i]);
  }
  __device__ __forceinline__ void from(const float (&v)[kN]) {
    T* t = reinterpret_cast<T*>(&q);
#pragma unroll
    for (int i = 0; i < kN; ++i) t[i] = from_f32<T>(v[i]);
  }
};
__device__ __forceinline__ float tl_word_max(const TlWord<float>& w) {
  float v[4];
  w.to(v);
  return tl_max_nan(tl_max_nan(v[0], v[1]), tl_max_nan(v[2], v[3]));
}
__device__ __forceinline__ float tl_word_max(const TlWord<__nv_bfloat16>& w) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w.q);
  const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
  return tl_max_nan(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float tl_word_max(const TlWord<__half>& w) {
  const __half2* h = reinterpret_cast<const __half2*>(&w.q);
  const __half2 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
  return tl_max_nan(__low2float(m), __high2float(m));
}

// A row as `head` single elements up to a 16-byte boundary, `words` words, and
// `tail` single elements. The single ones (at most 14) belong to the first CTA,
// one to a thread: the head's to threads 0.., the tail's to threads 16...
template <typename T>
struct TlRow {
  const T* p;
  int head, words, tail;
  __device__ __forceinline__ TlRow(const void* base, int64_t ld, long t, int V) {
    constexpr int n = TlWord<T>::kN;
    p = static_cast<const T*>(base) + t * ld;
    head = min(V, (int)((16 - ((uintptr_t)p & 15)) & 15) / (int)sizeof(T));
    words = (V - head) / n;
    tail = V - head - words * n;
  }
  // the thread's single element, -1 if it has none
  __device__ __forceinline__ int single(int rank, int V) const {
    const int i = threadIdx.x;
    if (rank != 0) return -1;
    return i < head ? i : (i >= 16 && i - 16 < tail ? V - tail + i - 16 : -1);
  }
};

// exp2 arguments of a row's elements relative to its maximum M: d = (x - M) c,
// c = log2(e) / tau. As one fused operation, x c - round(M c), it is off by the
// residual r = M c - round(M c), the same for all elements, which is put right in
// what the exponentials are multiplied with: 2^-r. Where M c is so large that r
// would not be small, the difference is taken first (`far`).
struct TlShift {
  float c, m, mc, r;
  bool far;
  __device__ __forceinline__ TlShift(float M, float scale) : c(scale), m(M) {
    mc = M * scale;
    far = !(fabsf(mc) < 65536.0f);
    r = far ? 0.0f : fmaf(M, scale, -mc);
  }
  template <bool FAR>
  __device__ __forceinline__ float arg(float x) const {
    return FAR ? (x - m) * c : fmaf(x, c, -mc);
  }
};

// Largest value, sum of exponentials relative to it and sum of those times their
// (base 2) arguments, of a part of a row.
struct TlPart {
  float m, s, d;
};

__device__ __forceinline__ void tl_merge(TlPart& a, float m, float c, float s, float d) {
  const float top = tl_max_nan(a.m, m);
  if (top == -INFINITY) return;  // (both empty)
  const float ua = fmaxf((a.m - top) * c, -1000.0f), ub = fmaxf((m - top) * c, -1000.0f);
  const float ea = tl_ex2(ua), eb = tl_ex2(ub);
  a.d = ea * (a.d + a.s * ua) + eb * (d + s * ub);
  a.s = ea * a.s + eb * s;
  a.m = top;
}

// ------------------------------------------------------ the teacher's entries
// Thread j has entry j. What is shared: the warps' largest value and sum, and
// how many of the CTA's entries are in its segment; then those, in order.
struct TlTeacher {
  float m[8], s[8], loss[8];
  int count[8];
  int id[kTlMaxEntries];
  float q[kTlMaxEntries], x[kTlMaxEntries];
};

struct TlEntry {
  int id;        // -1: none
  float v, x;    // value and the student's logit (where it was read)
  bool mine;     // in this CTA's segment
  uint32_t warp; // the warp's lanes whose entries are
};

__device__ __forceinline__ float tl_teacher_value(const TlArgs& a, size_t i) {
  return a.values_dtype == TM_F32    ? static_cast<const float*>(a.values)[i]
         : a.values_dtype == TM_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(a.values)[i])
                                     : to_f32(static_cast<const __half*>(a.values)[i]);
}

__device__ __forceinline__ void tl_entry_load(const TlArgs& a, long t, TlEntry& e) {
  e.id = -1, e.v = -INFINITY;
  if ((int)threadIdx.x < a.n) {
    const size_t i = (size_t)t * a.n + threadIdx.x;
    const long id = tl_index(a.ids, a.ids64, i);
    const float v = tl_teacher_value(a, i);
    if (id >= 0 && id < a.V) e.id = (int)id, e.v = v;
  }
}

// Whether element i is in the words [w0, w1) of a row or, for the first CTA, one of its single elements.
template <typename T>
__device__ __forceinline__ bool tl_mine(const TlRow<T>& row, int rank, int w0, int w1, int i, int V) {
  constexpr int n = TlWord<T>::kN;
  const int lo = rank == 0 ? 0 : row.head + min(row.words, w0) * n, hi = row.head + min(row.words, w1) * n;
  return (i >= lo && i < hi) || (rank == 0 && i >= V - row.tail && i < V);
}

// `all`: read every entry's logit, not only those of this CTA.
template <typename T>
__device__ __forceinline__ void tl_entry_start(const TlRow<T>& row, bool mine, bool all, float c, TlTeacher& te, TlEntry& e) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  e.mine = mine;
  e.x = e.mine || (all && e.id >= 0) ? to_f32(row.p[e.id]) : 0.0f;
  e.warp = __ballot_sync(0xFFFFFFFFu, e.mine);
  const float m = tl_warp_max(e.v);
  const float s = tl_warp_sum(m == -INFINITY ? 0.0f : tl_ex2((e.v - m) * c));
  if (lane == 0) te.m[warp] = m, te.s[warp] = s, te.count[warp] = __popc(e.warp);
}

// After a barrier: Q; the entry's q and ln q; this CTA's entries in te.
__device__ __forceinline__ float tl_entry_share(const TlArgs& a, long t, int warps, float c, TlTeacher& te, const TlEntry& e,
                                                float& q, float& lnq) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  TlPart p{-INFINITY, 0.0f, 0.0f};
  int before = 0;
  for (int w = 0; w < warps; ++w) {
    if (w * 32 >= a.n) break;
    tl_merge(p, te.m[w], c, te.s[w], 0.0f);
    if (w < warp) before += te.count[w];
  }
  float Q;
  if (p.m == -INFINITY) {
    Q = 0.0f, lnq = -INFINITY;
  } else if (a.teacher_lse) {
    const float lse = a.teacher_lse[t];
    Q = expf(p.m * a.inv_tau - lse) * p.s;
    lnq = e.v * a.inv_tau - lse;
  } else {
    Q = p.s * (1.0f / p.s);  // (1, or NaN)
    lnq = (e.v - p.m) * a.inv_tau - logf(p.s);
  }
  if (e.v == -INFINITY) lnq = -INFINITY;
  q = expf(lnq);
  if (e.mine) {
    const int i = before + __popc(e.warp & ((1u << lane) - 1));
    te.id[i] = e.id, te.q[i] = q, te.x[i] = e.x;
  }
  return Q;
}

// The gradient at this CTA's entries: the same token's q add up in their order.
template <typename T, typename P>
__device__ __forceinline__ void tl_entry_grad(const TlTeacher& te, int count, float g, float Q, T* out, P prob) {
  const int i = threadIdx.x;
  if (i >= count) return;
  const int id = te.id[i];
  float q = 0.0f;
  bool first = true;
  for (int x = 0; x < count; ++x)
    if (te.id[x] == id) {
      first = first && x >= i;
      q += te.q[x];
    }
  if (first) out[id] = from_f32<T>(g * (Q * prob(te.x[i]) - q));
}

// ------------------------------------------------------------- gradient pass
// out = e (A + B d), e = 2^d: with B = 0 the multiple A of the probability.
template <typename T, bool ENTROPY>
__device__ __forceinline__ float tl_grad_value(float x, const TlShift& sh, float A, float B) {
  float d = sh.far ? sh.arg<true>(x) : sh.arg<false>(x);
  if (ENTROPY) d = fmaxf(d, -1000.0f);  // (0 times infinity)
  return tl_ex2(d) * (ENTROPY ? fmaf(B, d, A) : A);
}

template <typename T, bool ENTROPY>
__device__ __forceinline__ void tl_grad_word(const TlWord<T>& w, T* out, bool vec, const TlShift& sh, float A, float B) {
  constexpr int n = TlWord<T>::kN;
  float v[n];
  w.to(v);
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = tl_grad_value<T, ENTROPY>(v[i], sh, A, B);
  TlWord<T> o;
  o.from(v);
  if (vec) {
    *reinterpret_cast<uint4*>(out) = o.q;
  } else {
    const T* e = reinterpret_cast<const T*>(&o.q);
#pragma unroll
    for (int i = 0; i < n; ++i) out[i] = e[i];
  }
}

// ------------------------------------------------------ the largest of a tile
// Threads of one lane number form 32 groups, over which neighbouring words are
// spread. The `top`-th largest of the groups' maxima is a bound that at least
// `top` elements reach. Those above it are collected (some 4 top of them for
// random data) and ranked by counting; if they are fewer than `top`, the first
// of those equal to it follow.
template <int NT>
struct TlTop {
  uint32_t group[NT];
  unsigned long long cand[kTlCandidates], list[kTlMaxTop], best[NT / 32];
  int n, warp[NT / 32];
};

// The k-th largest (k = 1..32) of the warp's values.
__device__ __forceinline__ uint32_t tl_kth(uint32_t v, int k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int o = size / 2; o; o /= 2) {
      const uint32_t u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
      const bool down = (lane & size) == 0 || size == 32, low = (lane & o) == 0;
      v = (low == down) ? max(u, v) : min(u, v);
    }
  return __shfl_sync(0xFFFFFFFFu, v, k - 1);
}

// Merges the tile's largest into to.list (sorted, 0 where there are fewer). The
// thread's elements: its words, and the single one of value xs where `single` is
// not -1; `mine`: the order of the largest (0: none). Ends without a barrier:
// to.list may be read after the next one.
template <typename T, int NT>
__device__ void tl_tile_top(TlTop<NT>& to, int top, bool first, const uint4* tile, int w0, int wn, const TlRow<T>& row,
                            int single, float xs, uint32_t mine) {
  constexpr int N = TlWord<T>::kN;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  to.group[tid] = mine;
  if (tid == 0) to.n = 0;
  __syncthreads();
  uint32_t g = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) g = max(g, to.group[w * 32 + lane]);
  uint32_t bound = tl_kth(g, top);
  const unsigned long long last = first ? 0ull : to.list[top - 1];
  const bool full = last != 0 && (uint32_t)(last >> 32) >= bound;  // (equals of a later tile come after those)
  if (full) bound = (uint32_t)(last >> 32);
  // words of the thread, in order: f(word's place in the tile, first index)
  auto words = [&](auto f) {
#pragma unroll 1
    for (int u = 0; u < kTlWords; ++u) {
      const int i = u * NT + tid;
      if (i < wn) f(i, row.head + (w0 + i) * N);
    }
  };
  auto put = [&](uint32_t o, int i) {
    const int at = atomicAdd(&to.n, 1);
    if (at < kTlCandidates) to.cand[at] = tl_key(o, i);
  };
  if (mine > bound) {
    words([&](int i, int at) {
      TlWord<T> w{tile[i]};
      if (tl_order(tl_word_max(w)) > bound) {
        const T* e = reinterpret_cast<const T*>(&tile[i]);
#pragma unroll 1
        for (int x = 0; x < N; ++x) {
          const uint32_t o = tl_order(to_f32(e[x]));
          if (o > bound) put(o, at + x);
        }
      }
    });
    if (single >= 0 && tl_order(xs) > bound) put(tl_order(xs), single);
  }
  __syncthreads();
  int n = to.n;
  if (n > kTlCandidates - kTlMaxTop) {
    // more than there is room for: the largest key below the last one, `top` times
    unsigned long long below = ~0ull;
    __syncthreads();
    for (n = 0; n < top; ++n) {
      unsigned long long best = 0;
      auto look = [&](uint32_t o, int i) {
        const unsigned long long k = tl_key(o, i);
        if (k < below && k > best) best = k;
      };
      words([&](int i, int at) {
        const T* e = reinterpret_cast<const T*>(&tile[i]);
#pragma unroll 1
        for (int x = 0; x < N; ++x) look(tl_order(to_f32(e[x])), at + x);
      });
      if (single >= 0) look(tl_order(xs), single);
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const unsigned long long b = __shfl_xor_sync(0xFFFFFFFFu, best, o);
        best = b > best ? b : best;
      }
      if (lane == 0) to.best[warp] = best;
      __syncthreads();
      for (int w = 0; w < NT / 32; ++w) best = to.best[w] > best ? to.best[w] : best;
      __syncthreads();
      if (tid == 0) to.cand[n] = best;
      below = best;
    }
    __syncthreads();
  } else if (n < top && !full && bound != 0) {
    // the first of the elements equal to the bound: the head's, the words' row by row, the tail's
    int need = top - n;
    for (int u = -1; u <= kTlWords && need > 0; ++u) {
      uint32_t same = 0;  // bits of the thread's elements
      int at = 0;
      if (u < 0 || u == kTlWords) {
        if (single >= 0 && (u < 0) == (tid < 16) && tl_order(xs) == bound) same = 1, at = single;
      } else if (u * NT + tid < wn) {
        at = row.head + (w0 + u * NT + tid) * N;
        const T* e = reinterpret_cast<const T*>(&tile[u * NT + tid]);
#pragma unroll
        for (int x = 0; x < N; ++x) same |= (uint32_t)(tl_order(to_f32(e[x])) == bound) << x;
      }
      int incl = __popc(same);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) to.warp[warp] = incl;
      __syncthreads();
      int before = incl - __popc(same), all = 0;
      for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += to.warp[w];
        all += to.warp[w];
      }
      while (same && before < need) {
        const int x = __ffs(same) - 1;
        same &= same - 1;
        to.cand[n + before++] = tl_key(bound, at + x);
      }
      n += min(all, need);
      need -= all;
      __syncthreads();
    }
  }
  // the earlier tiles' list, then ranks
  if (!first) {
    if (tid < top && to.list[tid]) to.cand[n + tid] = to.list[tid];
    int have = 0;
    for (int i = 0; i < top; ++i) have += to.list[i] != 0;
    n += have;
    __syncthreads();
  }
  if (tid < top) to.list[tid] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += NT) {
    const unsigned long long k = to.cand[i];
    int rank = 0;
    for (int x = 0; x < n; ++x) rank += to.cand[x] > k;
    if (rank < top) to.list[rank] = k;
  }
}

__device__ __forceinline__ uint32_t tl_map(const void* p, int rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return at;
}
__device__ __forceinline__ void tl_meet() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// (with their order among the reads of shared memory)
__device__ __forceinline__ void tl_copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void tl_copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void tl_copy_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

enum { kTlLogprobs = 0, kTlDistill = 1, kTlDistillGrad = 2 };

template <typename T, int NT, int MODE>
__global__ void __launch_bounds__(NT, NT == 256 ? 3 : 10) k_tl_rows(const TlArgs a) {
  constexpr int N = TlWord<T>::kN, W = kTlWords, TW = NT * W, NW = NT / 32;
  constexpr bool kEntropy = MODE == kTlLogprobs, kGrad = MODE == kTlDistillGrad;
  extern __shared__ uint4 tl_buf[];  // two tiles
  __shared__ __align__(16) float4 s_part[2][kTlCtas * NW];
  __shared__ unsigned long long s_lists[MODE == kTlLogprobs ? 2 * kTlCtas * kTlMaxTop : 1];
  __shared__ typename std::conditional<MODE == kTlLogprobs, TlTop<NT>, TlTeacher>::type sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = a.ctas == 1 ? 0 : (int)(blockIdx.x % a.ctas);
  const long step = gridDim.x / a.ctas;
  const float c = a.inv_tau * kLog2e;
  grid_wait();
  grid_launch();

  // words of tile p of the CTA's segment of a row: the first one's place, and how many
  auto tile_words = [&](const TlRow<T>& row, int p, int& w0) {
    w0 = rank * a.seg + p * TW;
    return max(0, min(min(row.words, (rank + 1) * a.seg) - w0, TW));
  };
  auto fetch = [&](long t, int p, int buf) {
    if (t < a.T && !(MODE != kTlLogprobs && a.mask && !a.mask[t])) {
      const TlRow<T> row(a.logits, a.ld, t, a.V);
      int w0;
      const int n = tile_words(row, p, w0);
      const T* src = row.p + row.head + (size_t)(w0 + tid) * N;
#pragma unroll
      for (int u = 0; u < W; ++u)
        if (u * NT + tid < n) tl_copy16(tl_buf + buf * TW + u * NT + tid, src + (size_t)u * NT * N);
    }
    tl_copy_commit();
  };
  // what a row needs besides, one row ahead
  TlEntry entry;
  long y = 0;
  float xs = 0.0f;
  auto ahead = [&](long t) {
    if (t >= a.T) return;
    if constexpr (MODE == kTlLogprobs)
      y = tl_index(a.targets, a.target64, t);
    else
      tl_entry_load(a, t, entry);
    const TlRow<T> row(a.logits, a.ld, t, a.V);
    const int i = row.single(rank, a.V);
    xs = i >= 0 ? to_f32(row.p[i]) : -INFINITY;
  };

  const int steps = a.tiles * (kGrad && a.tiles > 1 ? 2 : 1);  // tiles of a row that go through the buffers
  long t = blockIdx.x / a.ctas;
  int buf = 0, parity = 0;
  fetch(t, 0, 0);
  ahead(t);
  for (; t < a.T; t += step) {
    const bool masked = MODE != kTlLogprobs && a.mask && !a.mask[t];
    const TlRow<T> row(a.logits, a.ld, t, a.V);
    const int single = row.single(rank, a.V);
    const float x1 = xs;
    const TlEntry e0 = entry;
    const long target = y;
    T* out = kGrad ? static_cast<T*>(a.grad) + t * a.grad_ld : nullptr;
    if (masked) {  // (the same for the cluster)
      fetch(t + step, 0, buf ^ 1);
      ahead(t + step);
      buf ^= 1;
      if (kGrad) {
        TlWord<T> z;
        z.q = make_uint4(0, 0, 0, 0);
        for (int p = 0; p < a.tiles; ++p) {
          int w0;
          const int n = tile_words(row, p, w0);
          for (int i = tid; i < n; i += NT) {
            T* o = out + row.head + (size_t)(w0 + i) * N;
            if (a.vec_out)
              *reinterpret_cast<uint4*>(o) = z.q;
            else
              for (int x = 0; x < N; ++x) o[x] = from_f32<T>(0.0f);
          }
        }
        if (single >= 0) out[single] = from_f32<T>(0.0f);
      }
      if (rank == 0 && tid == 0) {
        a.loss[t] = 0.0f;
        if (a.stats) a.stats[2 * t] = a.stats[2 * t + 1] = 0.0f;
      }
      continue;
    }
    TlEntry e = e0;
    float xy = 0.0f;
    if constexpr (MODE == kTlLogprobs) {
      if (rank == 0 && tid == 0 && target >= 0 && target < a.V) xy = to_f32(row.p[target]);
    } else {
      tl_entry_start(row, tl_mine(row, rank, rank * a.seg, (rank + 1) * a.seg, e.id, a.V), rank == 0, c, sh, e);
    }
    TlPart part{-INFINITY, 0.0f, 0.0f};
    const int held = buf;  // (the row's only tile stays there)
    for (int p = 0; p < a.tiles; ++p) {
      if (p + 1 < steps)
        fetch(t, (p + 1) % a.tiles, buf ^ 1);
      else
        fetch(t + step, 0, buf ^ 1);
      tl_copy_wait<1>();
      int w0;
      const int n = tile_words(row, p, w0);
      const uint4* tile = tl_buf + buf * TW;
      buf ^= 1;
      TlWord<T> w[W];
      // (the head's single elements go with the first tile, the tail's with the last: tiles are in the row's order)
      const bool here = single >= 0 && p == (tid < 16 ? 0 : a.tiles - 1);
      const float xh = here ? x1 : -INFINITY;
      float m = xh;
#pragma unroll
      for (int u = 0; u < W; ++u)
        if (u * NT + tid < n) {
          w[u].q = tile[u * NT + tid];
          m = tl_max_nan(m, tl_word_max(w[u]));
        }
      const float wm = tl_warp_max(m);
      const TlShift shift(wm == -INFINITY ? 0.0f : wm, c);
      float s = 0.0f, dot = 0.0f;
      auto sums = [&](auto far) {
        auto add = [&](float x) {
          float d = shift.arg<decltype(far)::value>(x);
          if (kEntropy) d = fmaxf(d, -1000.0f);
          const float v = tl_ex2(d);
          s += v;
          if (kEntropy) dot = fmaf(v, d, dot);
        };
#pragma unroll
        for (int u = 0; u < W; ++u)
          if (u * NT + tid < n) {
            float v[N];
            w[u].to(v);
#pragma unroll
            for (int i = 0; i < N; ++i) add(v[i]);
          }
        add(xh);
      };
      if (shift.far)
        sums(std::true_type());
      else
        sums(std::false_type());
      // relative to the exact maximum
      if (kEntropy) dot -= shift.r * s;
      const float back = tl_ex2(-shift.r);
      tl_merge(part, wm, c, tl_warp_sum(s) * back, kEntropy ? tl_warp_sum(dot) * back : 0.0f);
      if constexpr (MODE == kTlLogprobs) {
        if (a.top)
          tl_tile_top<T, NT>(sh, a.top, p == 0, tile, w0, n, row, here ? single : -1, xh,
                             tid < n || here ? tl_order(m) : 0u);
      }
    }
    ahead(t + step);
    // every warp's part goes to all CTAs of the row
    __syncwarp();
    if (lane < a.ctas) {
      const uint32_t to = tl_map(&s_part[parity][rank * NW + warp], lane);
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"r"(to), "f"(part.m), "f"(part.s), "f"(part.d),
                   "f"(0.0f) : "memory");
    }
    if constexpr (MODE == kTlLogprobs) {
      if (a.top) {
        __syncthreads();
        if (tid < a.top) {
          const uint32_t to = tl_map(&s_lists[(parity * kTlCtas + rank) * a.top + tid], 0);
          asm volatile("st.shared::cluster.u64 [%0], %1;\n" ::"r"(to), "l"(sh.list[tid]) : "memory");
        }
      }
    }
    __syncwarp();
    tl_meet();
    TlPart all{-INFINITY, 0.0f, 0.0f};
    if (kGrad || rank == 0) {
      // (the same order for every warp of every CTA: lanes, then the tree)
      for (int i = lane; i < a.ctas * NW; i += 32) {
        const float4 v = s_part[parity][i];
        tl_merge(all, v.x, c, v.y, v.z);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const float m = __shfl_xor_sync(0xFFFFFFFFu, all.m, o), s = __shfl_xor_sync(0xFFFFFFFFu, all.s, o);
        const float d = __shfl_xor_sync(0xFFFFFFFFu, all.d, o);
        const bool low = (lane & o) == 0;  // (both lanes of a pair add in the same order)
        TlPart x{low ? all.m : m, low ? all.s : s, low ? all.d : d};
        tl_merge(x, low ? m : all.m, c, low ? s : all.s, low ? d : all.d);
        all = x;
      }
    }
    const bool none = all.m == -INFINITY;
    const float M = none ? 0.0f : all.m;
    const float lns = none ? -INFINITY : (all.m != all.m || all.m == INFINITY ? NAN : logf(all.s));
    auto logp = [&](float x) { return none ? -INFINITY : (x - M) * a.inv_tau - lns; };
    if constexpr (MODE == kTlLogprobs) {
      if (rank == 0 && tid == 0) {
        a.logprob[t] = target >= 0 && target < a.V ? logp(xy) : 0.0f;
        a.entropy[t] = none ? 0.0f : lns - all.d * kLn2 / all.s;
        a.stats[2 * t] = M;
        a.stats[2 * t + 1] = lns;
      }
      if (a.top && rank == 0) {
        const unsigned long long* l = s_lists + parity * kTlCtas * a.top;
        const int n = a.ctas * a.top;
        for (int i = tid; i < n; i += NT) {
          const unsigned long long k = l[i];
          int r = k ? 0 : kTlMaxTop;
          for (int x = 0; x < n; ++x) r += l[x] > k;
          if (r < a.top) {
            a.top_ids[t * a.top + r] = (int)~(uint32_t)k;
            a.top_logprobs[t * a.top + r] = logp(tl_value_of((uint32_t)(k >> 32)));
          }
        }
      }
    } else {
      float q, lnq;
      const float Q = tl_entry_share(a, t, NW, c, sh, e, q, lnq);
      if (rank == 0) {
        const float term = tl_warp_sum(e.id >= 0 && !(q == 0.0f) ? q * (lnq - logp(e.x)) : 0.0f);
        if (lane == 0) sh.loss[warp] = term;
      }
      const float g = kGrad ? a.grad_loss[t] * a.inv_tau : 0.0f;
      const TlShift shift(M, c);
      const float unit = none ? 0.0f : expf(-lns) * tl_ex2(-shift.r);  // p = 2^d unit
      if (kGrad) {
        const float A = g * Q * unit;
        for (int p = 0; p < a.tiles; ++p) {
          int at = held;
          if (a.tiles > 1) {
            if (p + 1 < a.tiles)
              fetch(t, p + 1, buf ^ 1);
            else
              fetch(t + step, 0, buf ^ 1);
            tl_copy_wait<1>();
            at = buf;
            buf ^= 1;
          }
          int w0;
          const int n = tile_words(row, p, w0);
#pragma unroll
          for (int u = 0; u < W; ++u)
            if (u * NT + tid < n) {
              TlWord<T> w{tl_buf[at * TW + u * NT + tid]};
              tl_grad_word<T, false>(w, out + row.head + (size_t)(w0 + u * NT + tid) * N, a.vec_out, shift, A, 0.0f);
            }
        }
        if (single >= 0) out[single] = from_f32<T>(tl_grad_value<T, false>(x1, shift, A, 0.0f));
      }
      int count = 0;  // (read here: after the barrier a warp may already be at the next row's)
      for (int w = 0; w < NW; ++w) count += w * 32 < a.n ? sh.count[w] : 0;
      __syncthreads();
      if (kGrad) {
        auto prob = [&](float x) { return unit * tl_ex2(shift.far ? shift.arg<true>(x) : shift.arg<false>(x)); };
        tl_entry_grad<T>(sh, count, g, Q, out, prob);
      }
      if (rank == 0 && tid == 0) {
        float loss = 0.0f;
        for (int w = 0; w < NW; ++w) loss += w * 32 < a.n ? sh.loss[w] : 0.0f;
        a.loss[t] = loss;
        if (a.stats) {
          a.stats[2 * t] = M;
          a.stats[2 * t + 1] = lns;
        }
      }
    }
    parity ^= 1;
  }
  tl_copy_wait<0>();
  __syncwarp();
  tl_meet();  // no CTA leaves while another may still write to it
}

// ------------------------------------------------------------------ backward
// One CTA for each NT * 8 words of a row.
template <typename T, int NT, bool ENTROPY, bool TEACHER>
__global__ void __launch_bounds__(NT) k_tl_backward(const TlArgs a) {
  constexpr int N = TlWord<T>::kN, W = kTlWords, NW = NT / 32;
  __shared__ typename std::conditional<TEACHER, TlTeacher, int>::type sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % a.ctas);
  const long t = blockIdx.x / a.ctas;
  const float c = a.inv_tau * kLog2e;
  grid_wait();
  grid_launch();
  const TlRow<T> row(a.logits, a.ld, t, a.V);
  const int single = row.single(rank, a.V);
  T* out = static_cast<T*>(a.grad) + t * a.grad_ld;
  const bool masked = TEACHER && a.mask && !a.mask[t];
  const int w0 = rank * NT * W, n = min(row.words - w0, NT * W);
  TlWord<T> w[W];
#pragma unroll
  for (int u = 0; u < W; ++u)
    if (u * NT + tid < n && !masked)
      w[u].q = *reinterpret_cast<const uint4*>(row.p + row.head + (size_t)(w0 + u * NT + tid) * N);
  const float x1 = single >= 0 && !masked ? to_f32(row.p[single]) : 0.0f;
  const float lns = masked ? 0.0f : a.stats[2 * t + 1];
  const TlShift shift(masked ? 0.0f : a.stats[2 * t], c);
  const float unit = masked || lns == -INFINITY ? 0.0f : expf(-lns) * tl_ex2(-shift.r);  // p = 2^d unit
  auto prob = [&](float x) { return unit * tl_ex2(shift.far ? shift.arg<true>(x) : shift.arg<false>(x)); };
  auto mine = [&](int i) { return tl_mine(row, rank, w0, w0 + NT * W, i, a.V); };
  float A = 0.0f, B = 0.0f, g, Q = 0.0f, xy = 0.0f;
  long y = -1;
  if constexpr (TEACHER) {
    if (!masked) {
      TlEntry e;
      tl_entry_load(a, t, e);
      tl_entry_start(row, mine(e.id), false, c, sh, e);
      __syncthreads();
      float q, lnq;
      Q = tl_entry_share(a, t, NW, c, sh, e, q, lnq);
      g = a.grad_loss[t] * a.inv_tau;
      A = g * Q * unit;
    }
  } else {
    y = tl_index(a.targets, a.target64, t);
    const bool has = y >= 0 && y < a.V;
    g = has && a.grad_logprob ? a.grad_logprob[t] * a.inv_tau : 0.0f;
    const float h = ENTROPY && a.grad_entropy ? a.grad_entropy[t] * a.inv_tau : 0.0f;
    if (tid == 0 && has && mine((int)y)) xy = to_f32(row.p[y]);
    // -g p - h p (ln p + H), ln p = ln 2 (d - r) - ln s
    A = -(g + h * ((-shift.r * kLn2 - lns) + (ENTROPY ? a.entropy[t] : 0.0f))) * unit;
    B = -h * kLn2 * unit;
    if (lns == -INFINITY) A = 0.0f;
    if (!has || !a.grad_logprob) y = -1;
    __syncthreads();  // (the target's logit is read before anybody writes there)
  }
#pragma unroll
  for (int u = 0; u < W; ++u)
    if (u * NT + tid < n) {
      if (masked) w[u].q = make_uint4(0, 0, 0, 0);
      tl_grad_word<T, ENTROPY>(w[u], out + row.head + (size_t)(w0 + u * NT + tid) * N, a.vec_out, shift, A, B);
    }
  if (single >= 0) out[single] = from_f32<T>(tl_grad_value<T, ENTROPY>(x1, shift, A, B));
  __syncthreads();
  if constexpr (TEACHER) {
    if (!masked) {
      int count = 0;
      for (int i = 0; i < NW; ++i) count += i * 32 < a.n ? sh.count[i] : 0;
      tl_entry_grad<T>(sh, count, g, Q, out, prob);
    }
  } else if (tid == 0 && y >= 0 && mine((int)y)) {
    out[y] = from_f32<T>(g + tl_grad_value<T, ENTROPY>(xy, shift, A, B));
  }
}

// CTAs of a row, threads and tiles. A short row takes one small CTA; a longer one
// as many as it takes to hold it, and with few rows as many as keep 8 KB each.
template <int NT>
void tl_shape(TlArgs& a, int es) {
  const long words = ((long)a.V * es + 15) / 16;
  int ctas = 1;
  while (ctas < kTlCtas && (words > (long)ctas * NT * kTlWords || ((long)a.T * ctas * 2 <= 152 && words / (2 * ctas) >= 512))) ctas *= 2;
  if (NT < 256) ctas = 1;
  a.ctas = ctas;
  a.seg = (int)((words + ctas - 1) / ctas);
  a.tiles = (a.seg + NT * kTlWords - 1) / (NT * kTlWords);
}

bool tl_small(const TlArgs& a, int es) {
  return ((long)a.V * es + 15) / 16 <= 64 * kTlWords && a.n <= 64;
}

template <typename T, int NT, int MODE>
cudaError_t tl_rows_launch(TlArgs a, cudaStream_t st) {
  auto kern = k_tl_rows<T, NT, MODE>;
  tl_shape<NT>(a, (int)sizeof(T));
  constexpr int smem = 2 * NT * kTlWords * 16;
  static OncePerDevice done;
  cudaError_t e = allow_smem(done, kern, smem);
  if (e != cudaSuccess) return e;
  const long most = 152L * (NT == 256 ? 3 : 10) / a.ctas;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(std::min<long>(a.T, most) * a.ctas));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)a.ctas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int MODE>
cudaError_t tl_rows(const TlArgs& a, int dtype, cudaStream_t st) {
  auto go = [&](auto elem) {
    using T = decltype(elem);
    return tl_small(a, sizeof(T)) ? tl_rows_launch<T, 64, MODE>(a, st) : tl_rows_launch<T, 256, MODE>(a, st);
  };
  return TM_BY_DTYPE(dtype, go);
}

template <bool ENTROPY, bool TEACHER>
cudaError_t tl_backward(TlArgs a, int dtype, cudaStream_t st) {
  auto go = [&](auto elem) {
    using T = decltype(elem);
    const bool small = tl_small(a, sizeof(T));
    const long words = ((long)a.V * (long)sizeof(T) + 15) / 16, per = (small ? 64 : 256) * kTlWords;
    a.ctas = (int)((words + per - 1) / per);
    const long ctas = (long)a.T * a.ctas;
    if (ctas >= 1L << 31) return cudaErrorInvalidConfiguration;
    if (small) return launch_after(k_tl_backward<T, 64, ENTROPY, TEACHER>, dim3((unsigned)ctas), 64, 0, st, a);
    return launch_after(k_tl_backward<T, 256, ENTROPY, TEACHER>, dim3((unsigned)ctas), 256, 0, st, a);
  };
  return TM_BY_DTYPE(dtype, go);
}

tm_status tl_check(const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t V, float temperature) {
  if (!dtype_ok(dtype)) return status_fail(TM_EINVAL, "dtype=%d is not a tm_dtype", dtype);
  if (T < 0) return status_fail(TM_EINVAL, "T=%d < 0", T);
  if (V < 1 || V > (1 << 30)) return status_fail(TM_EINVAL, "V=%d outside 1..%d", V, 1 << 30);
  if (ld < V) return status_fail(TM_EINVAL, "ld=%lld is less than V=%d", (long long)ld, V);
  if (!(temperature >= 1e-4f && temperature <= 1e4f)) return status_fail(TM_EINVAL, "temperature=%g outside 1e-4..1e4", temperature);
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

// The gradient's place.
void tl_grad_args(TlArgs& a, int dtype, void* grad, int64_t grad_ld) {
  const int64_t es = dtype_bytes(dtype);
  a.grad = grad, a.grad_ld = grad_ld;
  a.vec_out = (((uintptr_t)grad ^ (uintptr_t)a.logits) & 15) == 0 && (grad_ld - a.ld) * es % 16 == 0;
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
  const cudaError_t e = tl_rows<kTlLogprobs>(a, dtype, (cudaStream_t)stream);
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
  a.grad_logprob = grad_logprob, a.grad_entropy = grad_entropy;
  tl_grad_args(a, dtype, grad_logits, grad_ld);
  const cudaError_t e = grad_entropy ? tl_backward<true, false>(a, dtype, (cudaStream_t)stream)
                                     : tl_backward<false, false>(a, dtype, (cudaStream_t)stream);
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
  if (T == 0) return TM_OK;
  a.loss = loss, a.stats = stats;
  const cudaError_t e = tl_rows<kTlDistill>(a, dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "distillation");
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
  if (T == 0) return TM_OK;
  a.stats = const_cast<float*>(stats), a.grad_loss = grad_loss;
  tl_grad_args(a, dtype, grad_logits, grad_ld);
  const cudaError_t e = tl_backward<false, true>(a, dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "distillation backward");
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
  if (T == 0) return TM_OK;
  a.loss = loss, a.grad_loss = grad_loss;
  tl_grad_args(a, dtype, grad_logits, grad_ld);
  const cudaError_t e = tl_rows<kTlDistillGrad>(a, dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "distillation");
}

}  // extern "C"
