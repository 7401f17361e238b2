// Log probabilities of given tokens, and distillation from a teacher's largest
// logits (sm_103a). With u = l / tau, M = max l, s = ln sum exp((l - M) / tau):
//   log p_i = (l_i - M) / tau - s,   H = s - sum p_i (l_i - M) / tau
//   dl_i    = (g ([i = y] - p_i) - h p_i (log p_i + H)) / tau
//   loss    = sum_j q_j (ln q_j - log p_(i_j)),   dl_i = g (Q p_i - sum_(j: i_j = i) q_j) / tau
//
// Bound by memory: a row is read once, and its gradient written once.
//   k_tl_forward: a CTA goes through a row (few rows: a cluster shares one) in
//     tiles, the next one fetched while it works on this one. A thread reads only
//     words that it fetched itself (cp.async) and keeps its own maximum and sums, so
//     that no barrier stands between tiles; the threads' sums meet at the row's end.
//     (Words that may be among the largest are looked at by the whole warp, behind a
//     __syncwarp.)
//   k_tl_once: loss and gradient in one pass; a cluster holds the row in shared
//     memory between the sums and the gradient. Rows that are longer than that go
//     through it in tiles twice.
//   k_tl_backward: one CTA for each piece of a row.
// 4096 x 131072 bf16 (1.07 GB): log probabilities 157 to 165 us = 6.8 to 6.5 TB/s (five largest
// 182, twenty 237 to 242), distillation forward 172, gradients 314 and 334 to 342 us = 6.8 and 6.3 TB/s,
// loss and gradient in one pass 413 = 5.2. 8 rows: 3.4 us, with twenty largest 8.3.
#include <algorithm>
#include <cmath>

#include "elem.cuh"
#include "pdl.cuh"
#include "status.h"

namespace tmoe {

namespace {

constexpr int kTlMaxTop = 32;
constexpr int kTlMaxEntries = 256;
constexpr int kTlWords = 8;      // 16-byte words of a tile to a thread
constexpr int kTlCtas = 8;       // most CTAs of a cluster
constexpr float kLn2 = 0.6931471805599453f;

// log2(e) / tau is c, rounded down, and lo > 0 (so that -inf times either is
// -inf). The sums of the distillation's forward pass take both; those of the log
// probabilities take c and are put right by the arguments' mean, which they have;
// gradients take c (with both they took a tenth longer), which, c being off by
// less than 2^-23 of it, moves a p at 2^-10 of the largest by up to 2^-20 of it.
struct TlScale {
  float c, lo, rest;  // rest: lo / c
  float tau, inv;     // inv: 1 / tau, rounded
  // x / tau to the last bit or its neighbour (a tenth of a division's instructions)
  __device__ __forceinline__ float div(float x) const {
    const float q = x * inv;
    return fabsf(q) < INFINITY ? fmaf(fmaf(-q, tau, x), inv, q) : q;
  }
};

struct TlArgs {
  const void* logits;
  int64_t ld;
  int T, V;
  TlScale c;
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

// Two fp32 values that one instruction works on: the sums and gradients below are
// bound by their instructions, half as many with pairs.
struct TlPair {
  uint64_t v;
  __device__ __forceinline__ TlPair() {}
  __device__ __forceinline__ TlPair(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
  __device__ __forceinline__ float sum() const {
    float a, b;
    get(a, b);
    return a + b;
  }
  __device__ __forceinline__ TlPair ex2() const {
    float a, b;
    get(a, b);
    return TlPair(tl_ex2(a), tl_ex2(b));
  }
};
__device__ __forceinline__ TlPair tl_fma(TlPair a, TlPair b, TlPair c) {
  TlPair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ TlPair tl_add(TlPair a, TlPair b) {
  TlPair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ TlPair tl_mul(TlPair a, TlPair b) {
  TlPair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// 16 bytes of a row.
template <typename T>
struct TlWord {
  static constexpr int kN = 16 / (int)sizeof(T);
  uint4 q;
  __device__ __forceinline__ void to(float (&v)[kN]) const {
#pragma unroll
    for (int i = 0; i < kN; i += 2) pair(i / 2).get(v[i], v[i + 1]);
  }
  __device__ __forceinline__ uint32_t word(int i) const { return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w; }
  // elements 2 i and 2 i + 1
  __device__ __forceinline__ TlPair pair(int i) const {
    if constexpr (sizeof(T) == 4) return TlPair(__uint_as_float(word(2 * i)), __uint_as_float(word(2 * i + 1)));
    const uint32_t w = word(i);
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return TlPair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return TlPair(f.x, f.y);
  }
  __device__ __forceinline__ void set(int i, TlPair p) {
    float a, b;
    p.get(a, b);
    uint32_t* w = reinterpret_cast<uint32_t*>(&q);
    if constexpr (sizeof(T) == 4) {
      w[2 * i] = __float_as_uint(a), w[2 * i + 1] = __float_as_uint(b);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(a, b);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  __device__ __forceinline__ static TlWord none() {  // -inf throughout
    const uint32_t w = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __nv_bfloat16>::value ? 0xFF80FF80u : 0xFC00FC00u;
    return TlWord{make_uint4(w, w, w, w)};
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

// exp2 arguments of elements relative to a reference near their maximum m: with
// c = log2(e) / tau and the whole number w nearest to m c, d = x c - w is one fused
// operation with one rounding, and what belongs to different references differs by
// an exact power of two. BOTH: the same with c + lo, whose m lo, up to 128, belongs into w, or
// the maximum's own 2^d would be 0 or infinite. |w| below 2^30 is at most 32 (half a step of
// fp32 there) from the product, which is how large d gets at the maximum; beyond (`far`) the
// next value below it is 64 or more away: elements are either the maximum or do not count.
template <bool BOTH>
struct TlRef {
  TlScale c;
  float m, w;
  bool far;
  __device__ __forceinline__ TlRef(float max, const TlScale& scale) : c(scale) {
    m = max == -INFINITY ? 0.0f : max;
    w = rintf(BOTH ? fmaf(m, scale.c, m * scale.lo) : m * scale.c);
    far = !(fabsf(w) < 1073741824.0f);
  }
  __device__ __forceinline__ float near(float x) const {
    const float d = fmaf(x, c.c, -w);
    return BOTH ? fmaf(x, c.lo, d) : d;
  }
  __device__ __forceinline__ float arg(float x) const { return far ? (x == m ? 0.0f : x < m ? -1000.0f : NAN) : near(x); }
  // what the reference is below m
  __device__ __forceinline__ float above() const { return far ? 0.0f : near(m); }
};

// Largest value, sum of exponentials relative to its reference and sum of those
// times their (base 2) arguments, of a part of a row.
struct TlPart {
  float m, s, d;
  // to the reference of a larger maximum
  template <bool BOTH>
  __device__ __forceinline__ void raise(float top, const TlScale& c) {
    const TlRef<BOTH> a(m, c), b(top, c);
    const float u = m == top || m == -INFINITY ? 0.0f : fmaxf(a.far || b.far ? -1000.0f : a.w - b.w, -1000.0f);
    const float e = tl_ex2(u);
    d = e * fmaf(s, u, d);
    s *= e;
    m = top;
  }
};

// The parts of a warp's lanes (those of lanes past `n` are not looked at), the same for all lanes.
template <bool BOTH>
__device__ __forceinline__ TlPart tl_warp_merge(TlPart p, const TlScale& c) {
  const float top = tl_warp_max(p.m);
  p.raise<BOTH>(top, c);
  p.s = tl_warp_sum(p.s);
  p.d = tl_warp_sum(p.d);
  return p;
}

// ln sum exp of a row relative to its maximum, and sum p u' from its part. NaN
// where the row has a NaN or +inf; -inf where it has nothing.
template <bool BOTH>
__device__ __forceinline__ float tl_log_sum(const TlPart& p, const TlScale& c) {
  if (p.m == -INFINITY) return -INFINITY;
  if (p.m != p.m || p.m == INFINITY) return NAN;
  return logf(p.s) - TlRef<BOTH>(p.m, c).above() * kLn2;
}

// ------------------------------------------------------ the teacher's entries
// A thread has entries threadIdx.x + j NT, j < EPT.
constexpr int kTlStats = 5;  // of a distilled row: M, s, the teacher's maximum and its s (with teacher_lse: 0 and that), Q

struct TlTeacherWarps {
  float m[8], s[8], loss[8];  // by warp
};
struct TlTeacher : TlTeacherWarps {
  int count[2][8];            // by j and warp: entries in the CTA's part of the row
  int id[kTlMaxEntries];      // those, in their order
  float q[kTlMaxEntries], x[kTlMaxEntries];
};

struct TlEntry {
  int id;      // -1: none
  float v, x;  // value and the student's logit (where it was read)
};

__device__ __forceinline__ float tl_teacher_value(const TlArgs& a, size_t i) {
  return a.values_dtype == TM_F32    ? static_cast<const float*>(a.values)[i]
         : a.values_dtype == TM_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(a.values)[i])
                                     : to_f32(static_cast<const __half*>(a.values)[i]);
}

template <int NT, int EPT>
__device__ __forceinline__ void tl_entry_load(const TlArgs& a, long t, TlEntry (&e)[EPT]) {
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    e[j].id = -1, e[j].v = -INFINITY, e[j].x = 0.0f;
    const int k = threadIdx.x + j * NT;
    if (k < a.n) {
      const size_t i = (size_t)t * a.n + k;
      const long id = tl_index(a.ids, a.ids64, i);
      const float v = tl_teacher_value(a, i);
      if (id >= 0 && id < a.V) e[j].id = (int)id, e[j].v = v;
    }
  }
}

// Whether element i is in the words [w0, w1) of a row or, for the first CTA, one of its single elements.
template <typename T>
__device__ __forceinline__ bool tl_mine(const TlRow<T>& row, int rank, int w0, int w1, int i, int V) {
  constexpr int n = TlWord<T>::kN;
  const int lo = rank == 0 ? 0 : row.head + min(row.words, w0) * n, hi = row.head + min(row.words, w1) * n;
  return (i >= lo && i < hi) || (rank == 0 && i >= V - row.tail && i < V);
}

// What the teacher's distribution takes from each warp; before a barrier.
template <int NT, int EPT>
__device__ __forceinline__ void tl_teacher_part(const TlEntry (&e)[EPT], const TlScale& c, TlTeacherWarps& te) {
  float m = -INFINITY, s = 0.0f;
#pragma unroll
  for (int j = 0; j < EPT; ++j) m = tl_max_nan(m, e[j].v);
  m = tl_warp_max(m);
  if (m != -INFINITY) {  // (most warps have no entries)
#pragma unroll
    for (int j = 0; j < EPT; ++j) s += expf(c.div(e[j].v - m));
    s = tl_warp_sum(s);
  }
  if ((threadIdx.x & 31) == 0) te.m[threadIdx.x >> 5] = m, te.s[threadIdx.x >> 5] = s;
}

// ln q of an entry is (v - m) / tau - s.
struct TlTeacherSum {
  float m, s, Q;
};

// After the barrier.
template <int NT>
__device__ __forceinline__ TlTeacherSum tl_teacher_sum(const TlArgs& a, long t, const TlTeacherWarps& te) {
  // (a lane for a warp's part, the same in every eight lanes)
  const int w = threadIdx.x & 7;
  const float wm = w < NT / 32 ? te.m[w] : -INFINITY;
  float m = wm;
#pragma unroll
  for (int o = 4; o; o >>= 1) m = tl_max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float s = wm == -INFINITY ? 0.0f : te.s[w] * expf(a.c.div(wm - m));
#pragma unroll
  for (int o = 4; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (m == -INFINITY) return {0.0f, 0.0f, 0.0f};
  if (a.teacher_lse) {
    const float lse = a.teacher_lse[t];
    return {0.0f, lse, expf(a.c.div(m) - lse) * s};
  }
  return {m, logf(s), s == s ? 1.0f : s};  // (Q: 1, or NaN)
}

__device__ __forceinline__ float tl_ln_q(const TlEntry& e, const TlTeacherSum& k, const TlScale& c) {
  return e.v == -INFINITY ? -INFINITY : c.div(e.v - k.m) - k.s;
}

// This CTA's entries in te, in order: their numbers before a barrier ...
template <int EPT>
__device__ __forceinline__ void tl_entry_count(const bool (&mine)[EPT], TlTeacher& te, uint32_t (&lanes)[EPT]) {
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    lanes[j] = __ballot_sync(0xFFFFFFFFu, mine[j]);
    if ((threadIdx.x & 31) == 0) te.count[j][threadIdx.x >> 5] = __popc(lanes[j]);
  }
}
// ... and after it themselves; returns how many.
template <int NT, int EPT>
__device__ __forceinline__ int tl_entry_share(const TlEntry (&e)[EPT], const bool (&mine)[EPT], const uint32_t (&lanes)[EPT],
                                              const TlTeacherSum& k, const TlScale& c, TlTeacher& te) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int all = 0;
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    int at = all;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      const int n = te.count[j][w];
      at += w < warp ? n : 0;
      all += n;
    }
    if (mine[j]) {
      at += __popc(lanes[j] & ((1u << lane) - 1));
      te.id[at] = e[j].id, te.q[at] = expf(tl_ln_q(e[j], k, c)), te.x[at] = e[j].x;
    }
  }
  return all;
}

// The gradient at this CTA's entries: the same token's q add up in their order.
template <int NT, typename T, typename P>
__device__ __forceinline__ void tl_entry_grad(const TlTeacher& te, int count, float g, float Q, T* out, P prob) {
  for (int i = threadIdx.x; i < count; i += NT) {
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
}

// ------------------------------------------------------------- gradient pass
// out = e (A + B d), e = 2^d: with B = 0 the multiple A of the probability.
template <bool ENTROPY>
__device__ __forceinline__ float tl_grad_value(float x, const TlRef<false>& r, float A, float B) {
  float d = r.arg(x);
  if (ENTROPY) d = fmaxf(d, -1000.0f);  // (0 times infinity)
  return tl_ex2(d) * (ENTROPY ? fmaf(B, d, A) : A);
}

template <typename T, bool ENTROPY>
__device__ __forceinline__ void tl_grad_word(const TlWord<T>& w, T* out, bool vec, const TlRef<false>& r, float A, float B) {
  constexpr int n = TlWord<T>::kN;
  TlWord<T> o;
  if (!r.far) {
    const TlPair c(r.c.c, r.c.c), shift(-r.w, -r.w), a2(A, A), b2(B, B);
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      TlPair d = tl_fma(w.pair(i), c, shift);
      if (ENTROPY) {
        float x, y;
        d.get(x, y);
        d = TlPair(fmaxf(x, -1000.0f), fmaxf(y, -1000.0f));
      }
      o.set(i, tl_mul(d.ex2(), ENTROPY ? tl_fma(b2, d, a2) : a2));
    }
  } else {
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      float x, y;
      w.pair(i).get(x, y);
      o.set(i, TlPair(tl_grad_value<ENTROPY>(x, r, A, B), tl_grad_value<ENTROPY>(y, r, A, B)));
    }
  }
  if (vec) {
    *reinterpret_cast<uint4*>(out) = o.q;
  } else {
    const T* e = reinterpret_cast<const T*>(&o.q);
#pragma unroll
    for (int i = 0; i < n; ++i) out[i] = e[i];
  }
}

// p = 2^d unit
__device__ __forceinline__ float tl_unit(const TlRef<false>& r, float log_sum) {
  return log_sum == -INFINITY ? 0.0f : expf(-log_sum) * tl_ex2(-r.above());
}

// ------------------------------------------------------ the largest logits
// 64 groups of threads, over which neighbouring words are spread, keep their
// largest so far. The `top`-th largest of those is a bound that `top` elements
// reach; what reaches it is collected as the row goes by (some top log(tiles) of
// random values), and in the end ranked by counting. Where that is too many (equal
// values, or rows that rise), or fewer than `top` are above -inf, the row is
// gone through again.
template <int NT>
struct TlTop {
  static constexpr int kPer = NT == 32 ? 8 : 4, kRoom = kPer * NT;
  uint32_t group[64];
  unsigned long long cand[kRoom], list[kTlMaxTop], best[NT / 32];
  int n, left, warp[NT / 32];
};

constexpr uint32_t kTlOrderNone = 0x007FFFFFu;  // tl_order(-inf)

// The k-th largest (k = 1..32) of 64 values, the largest taken away until k are.
__device__ __forceinline__ uint32_t tl_kth(const uint32_t* g, int k) {
  const int lane = threadIdx.x & 31;
  uint32_t x = g[lane], y = g[lane + 32], m;
  for (;;) {
    m = __reduce_max_sync(0xFFFFFFFFu, max(x, y));
    k -= __popc(__ballot_sync(0xFFFFFFFFu, x == m)) + __popc(__ballot_sync(0xFFFFFFFFu, y == m));
    if (k <= 0 || m == 0) return m;
    x = x == m ? 0 : x;
    y = y == m ? 0 : y;
  }
}

template <int NT>
__device__ __forceinline__ void tl_put(TlTop<NT>& to, uint32_t order, int i) {
  const int at = atomicAdd(&to.n, 1);
  if (at < TlTop<NT>::kRoom) to.cand[at] = tl_key(order, i);
}

// A tile's elements that reach `least`, the n words of which a warp's lanes have NT
// apart, `first` the index of the first: lane by lane of the `hits` that have some, by
// the whole warp, a lane's 32 4-byte words at once (some 40 instructions a hit) ...
constexpr int kTlFewHits = 4;
template <typename T, int NT>
__device__ __forceinline__ void tl_collect_warp(TlTop<NT>& to, uint32_t hits, const uint4* tile, int n, uint32_t least, int first) {
  constexpr int N = TlWord<T>::kN;
  const int tid = threadIdx.x, lane = tid & 31;
  for (uint32_t hit = hits; hit; hit &= hit - 1) {
    const int src = (tid & ~31) + __ffs(hit) - 1, i = (lane >> 2) * NT + src;
    uint32_t k0 = 0, k1 = 0;  // orders of the lane's one or two elements
    if (i < n) {
      const uint32_t v = reinterpret_cast<const uint32_t*>(tile + i)[lane & 3];
      if constexpr (sizeof(T) == 4) {
        k0 = tl_order(__uint_as_float(v));
      } else {
        const T* h = reinterpret_cast<const T*>(&v);
        k0 = tl_order(to_f32(h[0])), k1 = tl_order(to_f32(h[1]));
      }
    }
    const bool one = k0 >= least, two = k1 >= least;
    const uint32_t b1 = __ballot_sync(0xFFFFFFFFu, one), b2 = __ballot_sync(0xFFFFFFFFu, two);
    int at = 0;
    if (lane == 0) at = atomicAdd(&to.n, __popc(b1) + __popc(b2));
    at = __shfl_sync(0xFFFFFFFFu, at, 0);
    const uint32_t before = (1u << lane) - 1;
    const int x = first + i * N + (lane & 3) * (4 / (int)sizeof(T));
    const int p1 = at + __popc(b1 & before), p2 = at + __popc(b1) + __popc(b2 & before);
    if (one && p1 < TlTop<NT>::kRoom) to.cand[p1] = tl_key(k0, x);
    if (two && p2 < TlTop<NT>::kRoom) to.cand[p2] = tl_key(k1, x + 1);
  }
}

// ... or, where most lanes have some, each lane its own words, of which it looks into those whose maximum does.
template <typename T, int NT, int W>
__device__ __noinline__ void tl_collect_lanes(TlTop<NT>& to, const uint4* tile, int n, uint32_t least, int first) {
  constexpr int N = TlWord<T>::kN;
  const int tid = threadIdx.x, lane = tid & 31;
  uint32_t words = 0;  // bits of those
#pragma unroll
  for (int u = 0; u < W; ++u)
    if (u * NT + tid < n) words |= (uint32_t)(tl_order(tl_word_max(TlWord<T>{tile[u * NT + tid]})) >= least) << u;
  while (__any_sync(0xFFFFFFFFu, words != 0)) {
    const int i = (__ffs(words) - 1) * NT + tid;
    uint32_t k[N], some = 0;
    if (words) {
      float v[N];
      TlWord<T>{tile[i]}.to(v);
#pragma unroll
      for (int x = 0; x < N; ++x) some |= (uint32_t)((k[x] = tl_order(v[x])) >= least) << x;
    }
    words &= words - 1;
    int incl = __popc(some);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    int at = 0;
    if (lane == 31) at = atomicAdd(&to.n, incl);
    at = __shfl_sync(0xFFFFFFFFu, at, 31) + incl - __popc(some);
#pragma unroll
    for (int x = 0; x < N; ++x)
      if (some >> x & 1) {
        if (at < TlTop<NT>::kRoom) to.cand[at] = tl_key(k[x], first + i * N + x);
        ++at;
      }
  }
}

// to.list: the largest of the n candidates. Needs a barrier before and after.
template <int NT>
__device__ __forceinline__ void tl_rank(TlTop<NT>& to, int n, int top) {
  for (int i = threadIdx.x; i < n; i += NT) {
    const unsigned long long k = to.cand[i];
    int rank = 0;
#pragma unroll 8
    for (int x = 0; x < n; ++x) rank += to.cand[x] > k;
    if (rank < top) to.list[rank] = k;
  }
}

// The same from the row itself, words [w0, w0 + wn) and the threads' single
// elements (`single` -1: none): the candidates above `bound`, of which at least
// `top` reach it, and the first of those equal to it.
template <typename T, int NT>
__device__ __noinline__ int tl_top_again(TlTop<NT>& to, int top, const TlRow<T> row, int w0, int wn, int single, float xs,
                                         uint32_t bound) {
  constexpr int N = TlWord<T>::kN;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint4* words = reinterpret_cast<const uint4*>(row.p + row.head) + w0;
  const int first = row.head + w0 * N;
  __syncthreads();
  if (tid == 0) to.n = 0;
  __syncthreads();
  for (int i = tid; i < wn; i += NT) {
    const TlWord<T> w{words[i]};
    if (tl_order(tl_word_max(w)) > bound) {
      float v[N];
      w.to(v);
#pragma unroll
      for (int x = 0; x < N; ++x)
        if (tl_order(v[x]) > bound) tl_put(to, tl_order(v[x]), first + i * N + x);
    }
  }
  if (single >= 0 && tl_order(xs) > bound) tl_put(to, tl_order(xs), single);
  __syncthreads();
  int n = to.n;
  if (n > TlTop<NT>::kRoom - top) {
    // more than there is room for: the largest key below the last one, `top` times
    unsigned long long below = ~0ull;
    for (n = 0; n < top; ++n) {
      unsigned long long best = 0;
      auto look = [&](float v, int i) {
        const unsigned long long k = tl_key(tl_order(v), i);
        if (k < below && k > best) best = k;
      };
      for (int i = tid; i < wn; i += NT) {
        const TlWord<T> w{words[i]};
        if (tl_order(tl_word_max(w)) < (uint32_t)(best >> 32)) continue;
        float v[N];
        w.to(v);
#pragma unroll
        for (int x = 0; x < N; ++x) look(v[x], first + i * N + x);
      }
      if (single >= 0) look(xs, single);
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
  } else {
    // the first of the elements equal to the bound: the head's, the words' in order, the tail's
    int need = top - n;
    const int rounds = (wn + NT - 1) / NT;
    for (int u = -1; u <= rounds && need > 0; ++u) {
      uint32_t same = 0;  // bits of the thread's elements
      int at = 0;
      if (u < 0 || u == rounds) {
        if (single >= 0 && (u < 0) == (tid < 16) && tl_order(xs) == bound) same = 1, at = single;
      } else if (u * NT + tid < wn) {
        at = first + (u * NT + tid) * N;
        const TlWord<T> w{words[u * NT + tid]};
        float v[N];
        w.to(v);
#pragma unroll
        for (int x = 0; x < N; ++x) same |= (uint32_t)(tl_order(v[x]) == bound) << x;
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
  __syncthreads();
  return n;
}

// At the end of a row (of the CTA's words of it): to.list, complete when this
// returns. Leaves `to` as the next row needs it behind a barrier.
template <typename T, int NT>
__device__ __forceinline__ void tl_top_finish(TlTop<NT>& to, int top, const TlRow<T>& row, int w0, int wn, int single, float xs) {
  constexpr int kPer = TlTop<NT>::kPer, kFew = 96;
  const int tid = threadIdx.x;
  __syncthreads();
  const int n = to.n;
  int left = n;
  if (n > kFew || n < top) {
    // those that reach the final bound
    const uint32_t bound = tl_kth(to.group, top);
    unsigned long long k[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) k[j] = tid + j * NT < n ? to.cand[tid + j * NT] : 0ull;
    if (tid == 0) to.left = 0;
    __syncthreads();
    left = 0;
    if (n <= TlTop<NT>::kRoom) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (k[j] != 0 && (uint32_t)(k[j] >> 32) >= bound) to.cand[atomicAdd(&to.left, 1)] = k[j];
      __syncthreads();
      left = to.left;
    }
    if (n > TlTop<NT>::kRoom || left < top) left = tl_top_again<T, NT>(to, top, row, w0, wn, single, xs, bound);
  }
  tl_rank(to, left, top);
  __syncthreads();
  if (tid == 0) to.n = 0;
  for (int i = tid; i < 64; i += NT) to.group[i] = 0;
}

__device__ __forceinline__ uint32_t tl_map(const void* p, int rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return at;
}
__device__ __forceinline__ void tl_push(void* p, int rank, const TlPart& v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"r"(tl_map(p, rank)), "f"(v.m), "f"(v.s), "f"(v.d), "f"(0.0f)
               : "memory");
}
__device__ __forceinline__ void tl_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tl_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
template <bool CLUSTER>
__device__ __forceinline__ void tl_meet() {
  if (CLUSTER) {
    tl_arrive();
    tl_wait();
  } else {
    __syncthreads();
  }
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

// A tile's words and a single element into a thread's part where the row's values
// are so large that exponents need care.
template <typename T, int NT, int W, bool ENTROPY>
__device__ __noinline__ TlPart tl_take_far(TlPart p, const uint4* tile, int n, float single, const TlScale& c) {
  constexpr int N = TlWord<T>::kN;
  const TlRef<!ENTROPY> r(p.m, c);
  auto add = [&](float x) {
    const float d = fmaxf(r.arg(x), -1000.0f), e = tl_ex2(d);  // (not 0 times infinity; a NaN shows in the maximum)
    p.s += e;
    if (ENTROPY) p.d = fmaf(e, d, p.d);
  };
  for (int u = threadIdx.x; u < min(n, W * NT); u += NT) {
    const TlWord<T> w{tile[u]};
    float v[N];
    w.to(v);
#pragma unroll
    for (int i = 0; i < N; ++i) add(v[i]);
  }
  if (single != -INFINITY) add(single);
  return p;
}

// (The distillation's sums, without ENTROPY, take c and lo, the others c.)
// Takes W words (of which the thread has those below n, NT apart) and a single
// element (-inf: none) into a thread's part; returns their maximum.
template <typename T, int NT, int W, bool ENTROPY>
__device__ __forceinline__ float tl_take_words(TlPart& p, const uint4* tile, int n, float single, const TlScale& c) {
  constexpr int N = TlWord<T>::kN;
  const int tid = threadIdx.x;
  TlWord<T> w[W];
  if (n >= NT * W) {
#pragma unroll
    for (int u = 0; u < W; ++u) w[u].q = tile[u * NT + tid];
  } else {
#pragma unroll
    for (int u = 0; u < W; ++u) {
      w[u] = TlWord<T>::none();
      if (u * NT + tid < n) w[u].q = tile[u * NT + tid];
    }
  }
  float m = single;
#pragma unroll
  for (int u = 0; u < W; ++u) m = tl_max_nan(m, tl_word_max(w[u]));
  const float top = tl_max_nan(p.m, m);
  if (!(top == p.m)) p.raise<!ENTROPY>(top, c);
  const TlRef<!ENTROPY> r(p.m, c);
  if (r.far) {
    p = tl_take_far<T, NT, W, ENTROPY>(p, tile, n, single, c);
    return m;
  }
  const TlPair c2(r.c.c, r.c.c), lo(r.c.lo, r.c.lo), shift(-r.w, -r.w);
  TlPair s(0.0f, 0.0f), dot(0.0f, 0.0f);  // (of this tile: short sums round less)
  auto add = [&](TlPair x) {
    TlPair d = tl_fma(x, c2, shift);
    if (!ENTROPY) d = tl_fma(x, lo, d);
    if (ENTROPY) {  // (not 0 times infinity)
      float a, b;
      d.get(a, b);
      d = TlPair(fmaxf(a, -1000.0f), fmaxf(b, -1000.0f));
    }
    const TlPair e = d.ex2();
    s = tl_add(s, e);
    if (ENTROPY) dot = tl_fma(e, d, dot);
  };
#pragma unroll
  for (int u = 0; u < W; ++u)
#pragma unroll
    for (int i = 0; i < N / 2; ++i) add(w[u].pair(i));
  if (single != -INFINITY) add(TlPair(single, -INFINITY));
  p.s += s.sum(), p.d += dot.sum();
  return m;
}

// (half the work where half of the words are not there)
template <typename T, int NT, int W, bool ENTROPY>
__device__ __forceinline__ float tl_take(TlPart& p, const uint4* tile, int n, float single, const TlScale& c) {
  return n > NT * W / 2 ? tl_take_words<T, NT, W, ENTROPY>(p, tile, n, single, c)
                        : tl_take_words<T, NT, W / 2, ENTROPY>(p, tile, n, single, c);
}

// The warps' parts of a row, by a warp: the same bits for every warp that merges them.
template <bool BOTH>
__device__ __forceinline__ TlPart tl_merge_parts(const float4* parts, int n, const TlScale& c) {
  TlPart p{-INFINITY, 0.0f, 0.0f};
  for (int i = threadIdx.x & 31; i < n; i += 32) {
    const float4 v = parts[i];
    TlPart x{v.x, v.y, v.z};
    const float top = tl_max_nan(p.m, x.m);
    if (!(top == p.m)) p.raise<BOTH>(top, c);
    if (!(top == x.m)) x.raise<BOTH>(top, c);
    p.s += x.s, p.d += x.d;
  }
  return tl_warp_merge<BOTH>(p, c);
}

// ------------------------------------------------------------------- forward
// CLUSTER: a row for each cluster; else a row for each CTA, and the next after it.
// KIND: distillation, log probabilities, or those and the largest (one kernel for the
// latter two took 170 us for 4096 x 131072 without any, not 157).
enum { kTlDistill = 0, kTlLogprobs = 1, kTlLargest = 2 };
template <typename T, int NT, int EPT, bool CLUSTER, int KIND>
__global__ void __launch_bounds__(NT, NT == 256 ? 2 : NT == 128 ? 6 : 18) k_tl_forward(const TlArgs a) {
  constexpr int N = TlWord<T>::kN, W = kTlWords, TW = NT * W, NW = NT / 32;
  extern __shared__ uint4 tl_buf[];  // two tiles
  __shared__ __align__(16) float4 s_part[2][CLUSTER ? kTlCtas * NW : NW];
  constexpr bool LOGPROBS = KIND != kTlDistill, TOP = KIND == kTlLargest;
  __shared__ unsigned long long s_lists[TOP && CLUSTER ? kTlCtas * kTlMaxTop : 1];
  __shared__ typename std::conditional<TOP, TlTop<NT>, TlTeacherWarps>::type sh[LOGPROBS ? 1 : 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = CLUSTER ? a.ctas : 1, rank = CLUSTER ? (int)(blockIdx.x % a.ctas) : 0;
  const long step = gridDim.x / ctas;
  const TlScale c = a.c;
  if constexpr (TOP) {
    for (int i = tid; i < 64; i += NT) sh[0].group[i] = 0;
    if (tid == 0) sh[0].n = 0;
    __syncthreads();
  }
  if (CLUSTER) tl_arrive();
  grid_wait();
  grid_launch();

  // words of tile p of the CTA's segment of a row: the first one's place, and how many
  auto tile_words = [&](const TlRow<T>& row, int p, int& w0) {
    w0 = rank * a.seg + p * TW;
    return max(0, min(min(row.words, (rank + 1) * a.seg) - w0, TW));
  };
  auto masked = [&](long t) { return !LOGPROBS && a.mask && !a.mask[t]; };
  auto fetch = [&](long t, int p, int buf) {
    if (t < a.T && !masked(t)) {
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
  TlEntry entry[EPT];
  long y = 0;
  float xs = 0.0f;
  auto ahead = [&](long t) {
    if (t >= a.T || masked(t)) return;
    if constexpr (LOGPROBS)
      y = tl_index(a.targets, a.target64, t);
    else
      tl_entry_load<NT>(a, t, entry);
    const TlRow<T> row(a.logits, a.ld, t, a.V);
    const int i = row.single(rank, a.V);
    xs = i >= 0 ? to_f32(row.p[i]) : -INFINITY;
  };

  long t = blockIdx.x / ctas;
  int buf = 0, parity = 0;
  // distillation: the warps' terms of a row are added up behind the next row's barrier, or after
  // the last one (with a barrier for each row's, 4096 x 131072 took 173 us)
  long open = -1;
  auto close = [&]() {
    if constexpr (!LOGPROBS) {
      if (tid == 0 && open >= 0) {
        float loss = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) loss += sh[parity ^ 1].loss[w];
        a.loss[open] = loss;
      }
    }
  };
  fetch(t, 0, 0);
  ahead(t);
  if (CLUSTER) tl_wait();  // (the first CTA runs: its shared memory may be written)
  for (; t < a.T; t += step) {
    if (masked(t)) {  // (the same for the cluster)
      fetch(t + step, 0, buf ^= 1);
      ahead(t + step);
      if (rank == 0 && tid == 0) a.loss[t] = 0.0f;
      if (rank == 0 && tid < kTlStats) a.stats[t * kTlStats + tid] = 0.0f;
      continue;
    }
    const TlRow<T> row(a.logits, a.ld, t, a.V);
    const int single = row.single(rank, a.V);
    const float x1 = xs;
    const long target = y;
    TlEntry e[EPT];
    float xy = 0.0f;
    if constexpr (LOGPROBS) {
      if (rank == 0 && tid == 0 && target >= 0 && target < a.V) xy = to_f32(row.p[target]);
    } else {
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        e[j] = entry[j];
        if (rank == 0 && e[j].id >= 0) e[j].x = to_f32(row.p[e[j].id]);
      }
      tl_teacher_part<NT>(e, c, sh[parity]);
    }
    TlPart part{-INFINITY, 0.0f, 0.0f};
    uint32_t most = 0, bound = 0;
    for (int p = 0; p < a.tiles; ++p) {
      if (p + 1 < a.tiles)
        fetch(t, p + 1, buf ^ 1);
      else
        fetch(t + step, 0, buf ^ 1);
      tl_copy_wait<1>();
      int w0;
      const int n = tile_words(row, p, w0);
      const uint4* tile = tl_buf + buf * TW;
      buf ^= 1;
      const bool here = single >= 0 && p == 0;
      const float m = tl_take<T, NT, W, LOGPROBS>(part, tile, n, here ? x1 : -INFINITY, c);
      if constexpr (TOP) {
        TlTop<NT>& to = sh[0];
        const uint32_t o = tid < n || here ? tl_order(m) : 0u;
        if (o > most) atomicMax(&to.group[tid & 63], most = o);
        if (p == 0) __syncthreads();
        // (later, with whatever the other warps have found so far: any bound of this row's will do)
        if ((p & (p - 1)) == 0) bound = tl_kth(to.group, a.top);
        const uint32_t least = max(bound, kTlOrderNone + 1);
        const uint32_t hits = __ballot_sync(0xFFFFFFFFu, o >= least);
        if (__popc(hits) > kTlFewHits) {
          tl_collect_lanes<T, NT, W>(to, tile, n, least, row.head + w0 * N);
        } else if (hits) {
          __syncwarp();  // (each lane has waited for its own copies: now all may read them)
          tl_collect_warp<T, NT>(to, hits, tile, n, least, row.head + w0 * N);
        }
        if (here && tl_order(x1) >= least) tl_put(to, tl_order(x1), single);
        __syncwarp();
      }
    }
    ahead(t + step);
    part = tl_warp_merge<!LOGPROBS>(part, c);
    if (lane == 0) {
      if (CLUSTER)
        tl_push(&s_part[parity][rank * NW + warp], 0, part);
      else
        s_part[parity][warp] = make_float4(part.m, part.s, part.d, 0.0f);
    }
    if constexpr (TOP) {
      const int w0 = rank * a.seg, wn = max(0, min(row.words, w0 + a.seg) - w0);
      tl_top_finish<T, NT>(sh[0], a.top, row, w0, wn, single, x1);
      if (CLUSTER) {
        if (tid < a.top)
          asm volatile("st.shared::cluster.u64 [%0], %1;\n" ::"r"(tl_map(&s_lists[rank * a.top + tid], 0)), "l"(sh[0].list[tid])
                       : "memory");
      }
    }
    tl_meet<CLUSTER>();
    close();
    if (rank == 0) {
      const TlPart all = tl_merge_parts<!LOGPROBS>(s_part[parity], ctas * NW, c);
      const bool none = all.m == -INFINITY;
      const float M = none ? 0.0f : all.m, raw = tl_log_sum<!LOGPROBS>(all, c);
      // the mean of ln 2 (x - M) c, by which the sum grows with c
      const float mean = LOGPROBS && !none ? (all.d / all.s - TlRef<false>(M, c).above()) * kLn2 : 0.0f;
      const float lns = LOGPROBS && !none ? fmaf(c.rest, mean, raw) : raw;
      auto logp = [&](float x) { return none ? -INFINITY : c.div(x - M) - lns; };
      if constexpr (LOGPROBS) {
        if (tid == 0) {
          a.logprob[t] = target >= 0 && target < a.V ? logp(xy) : 0.0f;
          a.entropy[t] = none ? 0.0f : raw - mean;  // (c's rounding moves both alike)
          a.stats[2 * t] = M;
          a.stats[2 * t + 1] = lns;
        }
        if constexpr (TOP) {
          auto store = [&](int r, unsigned long long k) {
            a.top_ids[t * a.top + r] = (int)~(uint32_t)k;
            a.top_logprobs[t * a.top + r] = logp(tl_value_of((uint32_t)(k >> 32)));
          };
          if (CLUSTER) {
            const int n = ctas * a.top;
            for (int i = tid; i < n; i += NT) {
              const unsigned long long k = s_lists[i];
              int r = 0;
#pragma unroll 8
              for (int x = 0; x < n; ++x) r += s_lists[x] > k;
              if (r < a.top) store(r, k);
            }
          } else if (tid < a.top) {
            store(tid, sh[0].list[tid]);
          }
        }
      } else {
        const TlTeacherSum k = tl_teacher_sum<NT>(a, t, sh[parity]);
        float term = 0.0f;
#pragma unroll
        for (int j = 0; j < EPT; ++j)
          if (e[j].id >= 0) {
            const float lnq = tl_ln_q(e[j], k, c), q = expf(lnq);
            if (!(q == 0.0f)) term += q * (lnq - logp(e[j].x));
          }
        term = tl_warp_sum(term);
        if (lane == 0) sh[parity].loss[warp] = term;
        open = t;
        if (tid == 0) {
          float* st = a.stats + t * kTlStats;
          st[0] = M, st[1] = lns, st[2] = k.m, st[3] = k.s, st[4] = k.Q;
        }
      }
    }
    parity ^= 1;
  }
  if (!LOGPROBS && open >= 0) {
    __syncthreads();
    close();
  }
  tl_copy_wait<0>();
}

// ------------------------------------------------------------------- one pass
template <typename T, int NT, int W, int EPT>
__global__ void __launch_bounds__(NT, NT == 256 ? 4 : NT == 128 ? 8 : 20) k_tl_once(const TlArgs a) {
  constexpr int N = TlWord<T>::kN, TW = NT * W, NW = NT / 32, kPart = 8;  // words of a thread taken at once
  extern __shared__ uint4 tl_buf[];  // one tile
  __shared__ __align__(16) float4 s_part[kTlCtas * NW];
  __shared__ TlTeacher te;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % a.ctas);
  const long t = blockIdx.x / a.ctas;
  const TlScale c = a.c;
  if (a.ctas > 1) tl_arrive();
  grid_wait();
  grid_launch();
  const TlRow<T> row(a.logits, a.ld, t, a.V);
  const int single = row.single(rank, a.V);
  T* out = static_cast<T*>(a.grad) + t * a.grad_ld;
  auto tile_words = [&](int p, int& w0) {
    w0 = rank * a.seg + p * TW;
    return max(0, min(min(row.words, (rank + 1) * a.seg) - w0, TW));
  };
  if (a.mask && !a.mask[t]) {  // (the same for the cluster)
    if (a.ctas > 1) tl_wait();
    for (int p = 0; p < a.tiles; ++p) {
      int w0;
      const int n = tile_words(p, w0);
      for (int i = tid; i < n; i += NT) {
        T* o = out + row.head + (size_t)(w0 + i) * N;
        if (a.vec_out)
          *reinterpret_cast<uint4*>(o) = make_uint4(0, 0, 0, 0);
        else
          for (int x = 0; x < N; ++x) o[x] = from_f32<T>(0.0f);
      }
    }
    if (single >= 0) out[single] = from_f32<T>(0.0f);
    if (rank == 0 && tid == 0) a.loss[t] = 0.0f;
    return;
  }
  auto fetch = [&](int p) {
    int w0;
    const int n = tile_words(p, w0);
    const T* src = row.p + row.head + (size_t)(w0 + tid) * N;
#pragma unroll
    for (int u = 0; u < W; ++u) {
      if (u * NT + tid < n) tl_copy16(tl_buf + u * NT + tid, src + (size_t)u * NT * N);
      if (u % kPart == kPart - 1) tl_copy_commit();
    }
    return n;
  };
  int n = fetch(0);
  TlEntry e[EPT];
  tl_entry_load<NT>(a, t, e);
  const float x1 = single >= 0 ? to_f32(row.p[single]) : -INFINITY;
  const float grad_loss = a.grad_loss[t];
  bool mine[EPT];
  uint32_t lanes[EPT];
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    mine[j] = tl_mine(row, rank, rank * a.seg, (rank + 1) * a.seg, e[j].id, a.V);
    if (mine[j] || (rank == 0 && e[j].id >= 0)) e[j].x = to_f32(row.p[e[j].id]);
  }
  tl_entry_count(mine, te, lanes);
  tl_teacher_part<NT>(e, c, te);
  TlPart part{-INFINITY, 0.0f, 0.0f};
  for (int p = 0; p < a.tiles; ++p) {
    if (p) n = fetch(p);
    const float xh = p == 0 ? x1 : -INFINITY;
    static_assert(W == 2 * kPart, "two parts");
    tl_copy_wait<1>();
    tl_take<T, NT, kPart, false>(part, tl_buf, n, xh, c);
    tl_copy_wait<0>();
    if (n > kPart * NT) tl_take<T, NT, kPart, false>(part, tl_buf + kPart * NT, n - kPart * NT, -INFINITY, c);
  }
  part = tl_warp_merge<true>(part, c);
  if (a.ctas > 1) tl_wait();  // (all CTAs run: their shared memory may be written)
  if (lane < a.ctas) tl_push(&s_part[rank * NW + warp], lane, part);
  if (a.ctas > 1)
    tl_meet<true>();
  else
    tl_meet<false>();
  const TlPart all = tl_merge_parts<true>(s_part, a.ctas * NW, c);
  const bool none = all.m == -INFINITY;
  const float M = none ? 0.0f : all.m, lns = tl_log_sum<true>(all, c);
  const TlTeacherSum k = tl_teacher_sum<NT>(a, t, te);
  const int count = tl_entry_share<NT>(e, mine, lanes, k, c, te);
  if (rank == 0) {
    float term = 0.0f;
#pragma unroll
    for (int j = 0; j < EPT; ++j)
      if (e[j].id >= 0) {
        const float lnq = tl_ln_q(e[j], k, c), q = expf(lnq);
        if (!(q == 0.0f)) term += q * (lnq - (none ? -INFINITY : c.div(e[j].x - M) - lns));
      }
    term = tl_warp_sum(term);
    if (lane == 0) te.loss[warp] = term;
  }
  const float g = grad_loss * c.inv;
  const TlRef<false> ref(M, c);
  const float unit = tl_unit(ref, lns), A = g * k.Q * unit;
  for (int p = a.tiles - 1; p >= 0; --p) {  // (the last tile is still here)
    if (p < a.tiles - 1) {
      fetch(p);
      tl_copy_wait<0>();
    }
    int w0;
    const int m = tile_words(p, w0);
#pragma unroll 8
    for (int u = 0; u < W; ++u)
      if (u * NT + tid < m)
        tl_grad_word<T, false>(TlWord<T>{tl_buf[u * NT + tid]}, out + row.head + (size_t)(w0 + u * NT + tid) * N, a.vec_out, ref, A, 0.0f);
  }
  if (single >= 0) out[single] = from_f32<T>(tl_grad_value<false>(x1, ref, A, 0.0f));
  __syncthreads();
  tl_entry_grad<NT>(te, count, g, k.Q, out, [&](float x) { return unit * tl_ex2(ref.arg(x)); });
  if (rank == 0 && tid == 0) {
    float loss = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) loss += te.loss[w];
    a.loss[t] = loss;
  }
}

// ------------------------------------------------------------------ backward
// One CTA for each NT * 8 words of a row.
template <typename T, int NT, int EPT, bool ENTROPY, bool TEACHER>
__global__ void __launch_bounds__(NT, NT == 256 ? 4 : 16) k_tl_backward(const TlArgs a) {
  constexpr int N = TlWord<T>::kN, W = kTlWords;
  __shared__ typename std::conditional<TEACHER, TlTeacher, int>::type sh;
  const int tid = threadIdx.x;
  const int rank = (int)(blockIdx.x % a.ctas);
  const long t = blockIdx.x / a.ctas;
  const TlScale c = a.c;
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
  auto mine = [&](int i) { return tl_mine(row, rank, w0, w0 + NT * W, i, a.V); };
  const float* st = a.stats + t * (TEACHER ? kTlStats : 2);
  const float lns = masked ? 0.0f : st[1];
  const TlRef<false> ref(masked ? 0.0f : st[0], c);
  const float unit = masked ? 0.0f : tl_unit(ref, lns);
  float A = 0.0f, B = 0.0f, g = 0.0f, Q = 0.0f, xy = 0.0f;
  long y = -1;
  int count = 0;
  if constexpr (TEACHER) {
    TlEntry e[EPT];
    bool own[EPT];
    uint32_t lanes[EPT];
    if (!masked) {
      tl_entry_load<NT>(a, t, e);
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        own[j] = mine(e[j].id);
        if (own[j]) e[j].x = to_f32(row.p[e[j].id]);
      }
      tl_entry_count(own, sh, lanes);
    }
    __syncthreads();  // (and the entries' logits are read before anybody writes there)
    if (!masked) {
      const TlTeacherSum k{st[2], st[3], st[4]};
      Q = k.Q;
      count = tl_entry_share<NT>(e, own, lanes, k, c, sh);
      g = a.grad_loss[t] * c.inv;
      A = g * Q * unit;
    }
  } else {
    y = tl_index(a.targets, a.target64, t);
    const bool has = y >= 0 && y < a.V && a.grad_logprob;
    g = has ? a.grad_logprob[t] * c.inv : 0.0f;
    const float h = ENTROPY ? a.grad_entropy[t] * c.inv : 0.0f;
    if (!has || !mine((int)y)) y = -1;
    if (tid == 0 && y >= 0) xy = to_f32(row.p[y]);
    // -g p - h p (ln p + H), ln p = ln 2 (d - above) - ln s
    A = -g * unit;
    if (ENTROPY) {
      A = -(g + h * ((-ref.above() * kLn2 - lns) + a.entropy[t])) * unit;
      B = -h * kLn2 * unit;
    }
    if (lns == -INFINITY) A = 0.0f;
    __syncthreads();  // (the target's logit is read before anybody writes there)
  }
#pragma unroll
  for (int u = 0; u < W; ++u)
    if (u * NT + tid < n) {
      if (masked) w[u].q = make_uint4(0, 0, 0, 0);
      tl_grad_word<T, ENTROPY>(w[u], out + row.head + (size_t)(w0 + u * NT + tid) * N, a.vec_out, ref, A, B);
    }
  if (single >= 0) out[single] = from_f32<T>(tl_grad_value<ENTROPY>(x1, ref, A, B));
  __syncthreads();
  if constexpr (TEACHER) {
    tl_entry_grad<NT>(sh, count, g, Q, out, [&](float x) { return unit * tl_ex2(ref.arg(x)); });
  } else if (tid == 0 && y >= 0) {
    out[y] = from_f32<T>(g + tl_grad_value<ENTROPY>(xy, ref, A, B));
  }
}

// ------------------------------------------------------------------ launches
long tl_words(const TlArgs& a, int es) { return ((long)a.V * es + 15) / 16; }

void tl_shape(TlArgs& a, int es, int ctas, int tile) {
  a.ctas = ctas;
  a.seg = (int)((tl_words(a, es) + ctas - 1) / ctas);
  a.tiles = std::max(1, (a.seg + tile - 1) / tile);
}

template <typename... P>
cudaError_t tl_launch(void (*kern)(P...), long ctas, int cluster, int threads, int smem, const TlArgs& a, cudaStream_t st) {
  if (ctas >= 1L << 31) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

// Lets a kernel have `smem` bytes, and its SM as much shared memory as there is:
// how many CTAs share one is what keeps the memory busy.
template <typename... P>
cudaError_t tl_allow(OncePerDevice& done, void (*kern)(P...), int smem) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return done(dev, [&] {
    const cudaError_t f = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    return f == cudaSuccess ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) : f;
  });
}

template <typename T, int NT, int EPT, bool CLUSTER, int KIND>
cudaError_t tl_forward_launch(TlArgs a, int ctas, int sms, cudaStream_t st) {
  auto kern = k_tl_forward<T, NT, EPT, CLUSTER, KIND>;
  constexpr int smem = 2 * NT * kTlWords * 16, resident = NT == 256 ? 2 : NT == 128 ? 6 : 18;
  static OncePerDevice done;
  const cudaError_t e = tl_allow(done, kern, smem);
  if (e != cudaSuccess) return e;
  tl_shape(a, (int)sizeof(T), ctas, NT * kTlWords);
  return tl_launch(kern, CLUSTER ? (long)a.T * ctas : std::min<long>(a.T, (long)sms * resident), ctas, NT, smem, a, st);
}

// Rows of up to 4 KB take a warp each (16384 x 1000 bf16: forward 34 us, with 128
// threads 56; x 2048: 37 and 56; x 4096 would be 54 and 56, but 101 and 82 with the
// five largest, and 90 and 74 for the distillation).
// Of more than 24 largest a warp's 32 groups give no useful bound (16384 x 1000, 24
// largest: 117 us, with 128 threads 123; 32 largest: 249 and 139).
bool tl_short(const TlArgs& a, long words) { return a.n <= 64 && words <= 256 && a.top <= 24; }

// Few rows take a cluster of CTAs of 256 threads each, twice as many of them as long as all
// clusters find a place at once: two CTAs an SM of clusters of two, three for two SMs of four, one
// of eight. log probabilities of 131072 bf16 and 20000, us:
//   16 rows   clusters of 8: 4.0, 3.4    of 4: 4.0, 2.9    (8 rows: 3.4, 3.1 and 4.0, 2.9; 16 x 200003: 5.5 and 6.0)
//   38        of 8: 7.0, 6.0             of 4: 5.1, 3.5
//   54        of 4: 5.2, 3.5             of 2: 5.7, 3.2    (54 x 200003: 8.1 and 8.9)
//   76        of 4: 8.0, 5.6             of 2: 5.7, 3.2
//   152       of 2: 8.3, 4.0             a row to a CTA of 128 threads: 11.2, 3.8
//   153       of 2: 12.0, 6.5            128 threads: 14.1, 4.3    (153 x 50021: 8.8 and 7.6)
//   304       of 2: 15.5, 7.9            128 threads: 14.5, 4.5
// Loss and gradient in one pass: 38 rows of 32768 7.4 with eight and 5.6 with four, 76 7.3 with four and 5.9 with two.
bool tl_more_ctas(const TlArgs& a, long words, int ctas, int sms) {
  const int halves = ctas == 1 ? 4 : ctas == 2 ? 3 : 2;  // CTAs for two SMs
  return 2L * ctas * a.T * 2 <= (long)sms * halves && words / (2 * ctas) >= 512;
}

// More rows: a CTA of 128 threads each, six of which share an SM.
template <int KIND>
cudaError_t tl_forward(const TlArgs& a, int dtype, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = current_sms(sms);
  if (e != cudaSuccess) return e;
  auto go = [&](auto elem) {
    using T = decltype(elem);
    const long words = tl_words(a, (int)sizeof(T));
    if (tl_short(a, words))
      return tl_forward_launch<T, 32, 2, false, KIND>(a, 1, sms, st);
    int ctas = 1;
    while (ctas < kTlCtas && tl_more_ctas(a, words, ctas, sms)) ctas *= 2;
    if (ctas > 1) return tl_forward_launch<T, 256, 1, true, KIND>(a, ctas, sms, st);
    return tl_forward_launch<T, 128, 2, false, KIND>(a, 1, sms, st);
  };
  return TM_BY_DTYPE(dtype, go);
}

template <typename T, int NT, int W, int EPT>
cudaError_t tl_once_launch(TlArgs a, int ctas, cudaStream_t st) {
  auto kern = k_tl_once<T, NT, W, EPT>;
  constexpr int smem = NT * W * 16;
  static OncePerDevice done;
  const cudaError_t e = tl_allow(done, kern, smem);
  if (e != cudaSuccess) return e;
  tl_shape(a, (int)sizeof(T), ctas, NT * W);
  // (no more than the segment has: up to four CTAs share an SM, not three. 4096 rows of
  // 20000: 90.5 -> 80 us, of 50021: 200 -> 182, of 131072, which fill it: 413)
  return tl_launch(kern, (long)a.T * ctas, ctas, NT, std::min(smem, a.seg * 16), a, st);
}

cudaError_t tl_once(const TlArgs& a, int dtype, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = current_sms(sms);
  if (e != cudaSuccess) return e;
  auto go = [&](auto elem) {
    using T = decltype(elem);
    const long words = tl_words(a, (int)sizeof(T));
    if (tl_short(a, words)) return tl_once_launch<T, 32, 16, 2>(a, 1, st);
    if (words <= 2048 && a.T > sms) return tl_once_launch<T, 128, 16, 2>(a, 1, st);
    int ctas = 1;
    while (ctas < kTlCtas && (words > (long)ctas * 4096 || tl_more_ctas(a, words, ctas, sms))) ctas *= 2;
    return tl_once_launch<T, 256, 16, 1>(a, ctas, st);
  };
  return TM_BY_DTYPE(dtype, go);
}

template <bool ENTROPY, bool TEACHER>
cudaError_t tl_backward(TlArgs a, int dtype, cudaStream_t st) {
  auto go = [&](auto elem) {
    using T = decltype(elem);
    const long words = tl_words(a, (int)sizeof(T));
    const bool small = words <= 64 * kTlWords && a.n <= 128;
    const long per = (small ? 64 : 256) * kTlWords;
    a.ctas = std::max(1, (int)((words + per - 1) / per));
    const long ctas = (long)a.T * a.ctas;
    if (ctas >= 1L << 31) return cudaErrorInvalidConfiguration;
    if (small) return launch_after(k_tl_backward<T, 64, 2, ENTROPY, TEACHER>, dim3((unsigned)ctas), 64, 0, st, a);
    return launch_after(k_tl_backward<T, 256, 1, ENTROPY, TEACHER>, dim3((unsigned)ctas), 256, 0, st, a);
  };
  return TM_BY_DTYPE(dtype, go);
}

void tl_temperature(TlArgs& a, float tau) {
  const double c = 1.4426950408889634 / tau;
  a.c.tau = tau;
  a.c.inv = 1.0f / tau;
  a.c.c = (float)c;
  if ((double)a.c.c > c) a.c.c = nextafterf(a.c.c, 0.0f);
  a.c.lo = std::max((float)(c - a.c.c), 1e-30f);
  a.c.rest = a.c.lo / a.c.c;
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
  a.logits = logits, a.ld = ld, a.T = T, a.V = V;
  tl_temperature(a, temperature);
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
  a.logits = logits, a.ld = ld, a.T = T, a.V = V;
  tl_temperature(a, temperature);
  a.targets = targets, a.target64 = target_bytes == 8, a.top = top;
  a.logprob = logprob, a.entropy = entropy, a.stats = stats, a.top_ids = top_ids, a.top_logprobs = top_logprobs;
  const cudaError_t e = top > 0 ? tl_forward<kTlLargest>(a, dtype, (cudaStream_t)stream)
                                : tl_forward<kTlLogprobs>(a, dtype, (cudaStream_t)stream);
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
  a.logits = logits, a.ld = ld, a.T = T, a.V = V;
  tl_temperature(a, temperature);
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
  const cudaError_t e = tl_forward<kTlDistill>(a, dtype, (cudaStream_t)stream);
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
  const cudaError_t e = tl_once(a, dtype, (cudaStream_t)stream);
  return e == cudaSuccess ? TM_OK : status_cuda(e, "distillation");
}

}  // extern "C"
