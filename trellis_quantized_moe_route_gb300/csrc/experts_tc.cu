// Products by expert with 16-bit weights on the tensor cores (sm_103a), for rows
// that TMA can read (addresses and strides of 16 bytes).
//
// One kernel for the three products; D = A B^T with 128 rows of A as the M side
// (TMEM lanes) and up to 256 rows of B as the N side (columns):
//   forward  D[n, r]  A = W_e [n, k]           B = rows of x by route     contraction k
//   grad_x   D[k, r]  A = W_e^T (M contiguous) B = rows of dy             contraction n
//   grad_w   D[n, k]  A = dy^T (M contiguous)  B = x^T (N contiguous)     contraction over the expert's routes
// With the routes as columns, a block of them may have any multiple of 16 rows,
// so that experts with few routes waste little, and the weights, which bound
// these products by their bytes, are read by every block once. Rows are fetched
// where they lie, by the plan's order (gather copies of four rows): there is no
// sorted copy of x or dy, and results go straight to route order.
#include <algorithm>

#include "elem.cuh"
#include "experts.h"
#include "mxfp4_mma.cuh"
#include "status.h"
#include "tensor_map.h"
#include "tile_store.cuh"

namespace tmoe {

namespace {

constexpr int kEtEpiWarps = 8;
constexpr int kEtThreads = (kEtEpiWarps + 2) * 32;
constexpr int kEtMaxRing = 12;
constexpr uint32_t kEtSmem = 224 * 1024;
constexpr uint32_t kEtABytes = 128 * 128;      // 128 rows of 64 elements, or 64 of 128
constexpr uint32_t kEtGroup = 64 * 128;        // 64 rows of 64 elements (contiguous along M or N)
constexpr uint32_t kEtStoreBytes = 16 * 256;   // for four epilogue warps
constexpr int kEtMaxGroups = 257 + 1;

struct EtArgs {
  CUtensorMap amap, bmap;
  int E, R, M, depth;       // M: output channels; depth: contraction (forward, grad_x)
  int cols;                 // grad_w: columns of dW
  int bn;                   // most columns of a unit
  int bf16, per_route, vec; // vec: results can be stored in 16-byte words
  const int32_t *order, *offsets;
  void* out;
  uint32_t* flags;
};

struct EtBars {
  uint64_t full[kEtMaxRing], empty[kEtMaxRing];
  uint64_t acc_full[2], acc_empty[2];
};

// The groups of routes: where each begins, and its first block.
struct EtGroups {
  int off[kEtMaxGroups], first[kEtMaxGroups];
};

struct EtUnit {
  int expert, tile, slot0, rows, depth;  // rows: columns of D; grad_w: tile of M, slot0 the first route, col0
  int col0;
};

template <int MODE>
__device__ __forceinline__ EtUnit et_unit(const EtArgs& a, const EtGroups& g, int u, int units, FastDiv tiles, FastDiv ctiles) {
  EtUnit m;
  const int v = min(u, units - 1);
  int b = (int)tiles.div((uint32_t)v);
  m.tile = v - b * (int)tiles.d;
  if (MODE == kExGradW) {
    m.expert = (int)ctiles.div((uint32_t)b);
    m.col0 = (b - m.expert * (int)ctiles.d) * a.bn;
    m.rows = min(a.bn, a.cols - m.col0);
    m.slot0 = g.off[m.expert];
    m.depth = g.off[m.expert + 1] - m.slot0;
  } else {
    int n = 0;
    for (int e = (threadIdx.x & 31); e <= a.E; e += 32) n += g.first[e] <= b;
    m.expert = __reduce_add_sync(0xFFFFFFFFu, n) - 1;
    const int r0 = (b - g.first[m.expert]) * a.bn;
    m.slot0 = g.off[m.expert] + r0;
    m.rows = min(a.bn, g.off[m.expert + 1] - m.slot0);
    m.depth = m.expert == a.E ? 0 : a.depth;  // (routes of no expert: zeros)
    m.col0 = 0;
  }
  return m;
}

__device__ __forceinline__ int et_up16(int n) { return (n + 15) & ~15; }

__device__ __forceinline__ void et_tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n"
               ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
// Four rows of 64 elements, from column x.
__device__ __forceinline__ void et_gather4(uint32_t dst, const CUtensorMap* map, int x, const int (&r)[4], uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n"
      ::"r"(dst), "l"(map), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar) : "memory");
}

// Descriptor of an operand that is contiguous along M or N, 128-byte swizzled:
// 64 of those by 8 of the contraction are an atom of 1024 bytes; atoms follow each
// other along the contraction, and groups of 64 along M or N are kEtGroup apart. A step
// of 16 advances by two atoms.
__device__ __forceinline__ uint64_t et_desc_mn(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)(kEtGroup >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}

// 16-bit operands, fp32 accumulator, M = 128.
template <int MODE>
__device__ __forceinline__ uint32_t et_idesc(int bf16, int n) {
  return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((MODE != kExForward ? 1u : 0u) << 15) |
         ((MODE == kExGradW ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// (returns the stages it loaded)
template <int MODE>
__device__ int et_loader(const EtArgs& a, const EtGroups& g, EtBars& B, uint32_t base, uint32_t stage_bytes, int ring, int units,
                         FastDiv tiles, FastDiv ctiles, FastDiv topk, volatile int* abort) {
  const int lane = threadIdx.x & 31;
  const bool lead = mx_elect();
  const uint32_t bar0 = smem_u32(&B.full[0]);
  MxRing r;
  int it = 0;
  auto source = [&](int route) { return a.per_route ? route : (int)topk.div((uint32_t)route); };
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const EtUnit m = et_unit<MODE>(a, g, u, units, tiles, ctiles);
    const int stages = (m.depth + 63) / 64;
    if (stages == 0) continue;
    int q[2][4];
    if (MODE != kExGradW) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int route = __ldg(a.order + m.slot0 + min((lane + 32 * h) * 4 + i, m.rows - 1));  // (past the last row: any)
          q[h][i] = MODE == kExForward ? source(route) : route;
        }
    }
    const int quads = et_up16(m.rows) / 4;
    auto routes = [&](int s, int (&to)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) to[i] = __ldg(a.order + m.slot0 + min(s * 64 + (lane & 15) * 4 + i, m.depth - 1));
    };
    if (MODE == kExGradW) routes(0, q[0]);
    for (int s = 0; s < stages; ++s, ++it, r.next(ring)) {
      if (it >= ring && !mx_wait_warp(&B.empty[r.slot], r.phase ^ 1, abort, kMxWaitNs)) return it;
      const uint32_t st = base + (uint32_t)r.slot * stage_bytes, bar = bar0 + (uint32_t)r.slot * 8;
      if (MODE == kExGradW) {
        const int n = et_up16(min(64, m.depth - s * 64)), groups = (m.rows + 63) / 64;
        const int agroups = a.M - m.tile * 128 > 64 ? 2 : 1;  // (what lies past the last channel is not stored)
        if (lead) mx_expect(bar, (uint32_t)(n * 128 * (agroups + groups)));
        __syncwarp();
        int x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = source(q[0][i]);
        const int quad = lane & 15, half = lane >> 4;
        if (quad * 4 < n) {
          if (half < agroups) et_gather4(st + half * kEtGroup + quad * 512, &a.amap, m.tile * 128 + half * 64, q[0], bar);
          for (int c = half; c < groups; c += 2)
            et_gather4(st + kEtABytes + c * kEtGroup + quad * 512, &a.bmap, m.col0 + c * 64, x, bar);
        }
        if (s + 1 < stages) routes(s + 1, q[0]);
      } else {
        if (lead) {
          mx_expect(bar, kEtABytes + (uint32_t)quads * 512);
          if (MODE == kExForward) {
            et_tma_3d(st, &a.amap, s * 64, m.tile * 128, m.expert, bar);
          } else {
            et_tma_3d(st, &a.amap, m.tile * 128, s * 64, m.expert, bar);
            et_tma_3d(st + kEtGroup, &a.amap, m.tile * 128 + 64, s * 64, m.expert, bar);
          }
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (lane + 32 * h < quads) et_gather4(st + kEtABytes + (uint32_t)(lane + 32 * h) * 512, &a.bmap, s * 64, q[h], bar);
      }
    }
  }
  return it;
}

// (returns the stages whose MMAs it issued)
template <int MODE>
__device__ int et_issuer(const EtArgs& a, const EtGroups& g, EtBars& B, uint32_t base, uint32_t stage_bytes, int ring, int units,
                         FastDiv tiles, FastDiv ctiles, uint32_t tmem, volatile int* abort) {
  const int lane = threadIdx.x & 31;
  const bool lead = mx_elect();
  MxRing r;
  int it = 0, nu = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const EtUnit m = et_unit<MODE>(a, g, u, units, tiles, ctiles);
    const int stages = (m.depth + 63) / 64;
    if (stages == 0) continue;
    const int buf = nu & 1;
    if (nu >= 2 && !mx_wait_warp(&B.acc_empty[buf], ((nu >> 1) - 1) & 1, abort, kMxWaitNs)) return it;
    ++nu;
    tc_fence_after();
    const uint32_t idesc = et_idesc<MODE>(a.bf16, et_up16(m.rows)), d = tmem + (uint32_t)(buf * a.bn);
    for (int s = 0; s < stages; ++s, ++it, r.next(ring)) {
      if (!mx_wait_warp(&B.full[r.slot], r.phase, abort, kMxWaitNs)) return it;
      const uint32_t st = base + (uint32_t)r.slot * stage_bytes;
      const int left = min(64, m.depth - s * 64), steps = (left + 15) / 16;
      if (MODE == kExGradW && (left & 15)) {
        // rows past the last route, which the copies filled with some row, become zeros in both operands
        const int groups = 2 + (m.rows + 63) / 64, n = (et_up16(left) - left) * 8;
        for (int i = lane; i < groups * n; i += 32) {
          const int c = i / n, w = i - c * n;
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};\n" ::"r"(st + c * kEtGroup + left * 128 + w * 16), "r"(0) : "memory");
        }
        fence_proxy_async();
        __syncwarp();
      }
      tc_fence_after();
      const uint64_t ad = MODE == kExForward ? smem_desc_sw128(st) : et_desc_mn(st);
      const uint64_t bd = MODE == kExGradW ? et_desc_mn(st + kEtABytes) : smem_desc_sw128(st + kEtABytes);
      constexpr uint64_t sa = MODE == kExForward ? 2 : 128, sb = MODE == kExGradW ? 128 : 2;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < steps && lead) tc_mma_f16(d, ad + k * sa, bd + k * sb, idesc, s > 0 || k > 0 ? 1u : 0u);
      if (lead) tc_commit(&B.empty[r.slot]);
    }
    if (lead) tc_commit(&B.acc_full[buf]);
  }
  return it;
}

// 32 columns of dW of a thread's row.
template <typename O>
__device__ __forceinline__ void et_store_row(const float (&y)[32], O* __restrict__ out, int cols, bool vec) {
  constexpr int n = 16 / (int)sizeof(O);
  if (vec) {
#pragma unroll
    for (int c = 0; c < 32; c += n) {
      uint4 q;
      O* e = reinterpret_cast<O*>(&q);
#pragma unroll
      for (int i = 0; i < n; ++i) e[i] = from_f32<O>(y[c + i]);
      if (c < cols) *reinterpret_cast<uint4*>(out + c) = q;  // (cols is a multiple of n)
    }
  } else {
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (c < cols) out[c] = from_f32<O>(y[c]);
  }
}

template <int MODE, typename O>
__device__ void et_epilogue(const EtArgs& a, const EtGroups& g, EtBars& B, int units, FastDiv tiles, FastDiv ctiles, uint32_t tmem,
                            unsigned char* stage, volatile int* abort) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quarter = warp & 3, part = warp >> 2;
  const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
  O* out = static_cast<O*>(a.out);
  constexpr int kStep = kEtEpiWarps / 4 * 32;
  int nu = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const EtUnit m = et_unit<MODE>(a, g, u, units, tiles, ctiles);
    const bool some = m.depth > 0;
    const int buf = nu & 1, n = m.tile * 128 + quarter * 32 + lane;
    if (some) {
      const bool full = mx_wait_warp(&B.acc_full[buf], (nu >> 1) & 1, abort, kMxWaitNs);
      // the warps of a part meet at its barrier while they store: they go on together or not at all
      if (!mx_vote_part(full, 1 + part)) return;
      ++nu;
      tc_fence_after();
    }
    const uint32_t d = tmem + lane_base + (uint32_t)(buf * a.bn);
    for (int c0 = part * 32; c0 < m.rows; c0 += kStep) {
      float y[32];
      int row = 0;
      if (MODE != kExGradW) row = __ldg(a.order + m.slot0 + min(c0 + lane, m.rows - 1));
      if (some) {
        uint32_t v[32];
        tmem_ld32(d + c0, v);
        tmem_ld_wait();
        reg_fence32(v);
#pragma unroll
        for (int c = 0; c < 32; ++c) y[c] = __uint_as_float(v[c]);
      } else {
#pragma unroll
        for (int c = 0; c < 32; ++c) y[c] = 0.0f;
      }
      if (MODE == kExGradW) {
        if (n < a.M)
          et_store_row<O>(y, out + ((size_t)m.expert * a.M + n) * a.cols + m.col0 + c0, m.rows - c0, a.vec);
      } else if (sizeof(O) == 2 && a.vec) {
        mx_store32_words<O>(y, out, row, m.rows - c0, m.tile, a.M, stage + part * kEtStoreBytes, 1 + part);
      } else {
        mx_store32<O>(y, out, row, m.rows - c0, n, a.M);
      }
    }
    if (some) {
      tc_fence_before();
      if (lane == 0) mbar_arrive(&B.acc_empty[buf]);
    }
    __syncwarp();
  }
}

template <int MODE, typename O>
__global__ void __launch_bounds__(kEtThreads, 1) k_ex_tc(const __grid_constant__ EtArgs a, int ring, FastDiv tiles, FastDiv ctiles,
                                                         FastDiv topk) {
  extern __shared__ unsigned char et_smem_raw[];
  __shared__ __align__(8) EtBars bars;
  __shared__ EtGroups groups;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort;
  unsigned char* smem = et_smem_raw + ((1024u - (smem_u32(et_smem_raw) & 1023u)) & 1023u);
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ring; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], kEtEpiWarps);
    }
    s_abort = 0;
    mbar_fence_init();
  }
  if (threadIdx.x == kEtEpiWarps * 32) {
    mx_prefetch_map(&a.amap);
    mx_prefetch_map(&a.bmap);
  }
  if (warp == 0) tmem_alloc(&tmem_slot, 512);
  grid_wait();
  grid_launch();
  for (int e = threadIdx.x; e <= a.E; e += kEtThreads) groups.off[e] = a.offsets[e];
  if (threadIdx.x == 0) groups.off[a.E + 1] = a.R;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (MODE != kExGradW && warp == 0) {  // blocks before each group
    int run = 0;
    for (int e0 = 0; e0 <= a.E; e0 += 32) {
      const int e = e0 + lane;
      const int v = e <= a.E ? (groups.off[e + 1] - groups.off[e] + a.bn - 1) / a.bn : 0;
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += w;
      }
      if (e <= a.E) groups.first[e] = run + incl - v;
      run += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (lane == 0) groups.first[a.E + 1] = run;
  }
  __syncthreads();
  const uint32_t tmem = tmem_slot, base = smem_u32(smem), stage_bytes = kEtABytes + (uint32_t)a.bn * 128;
  const int units = MODE == kExGradW ? a.E * (int)ctiles.d * (int)tiles.d : groups.first[a.E + 1] * (int)tiles.d;
  volatile int* abort = &s_abort;
  int loaded = 0, issued = 0;
  if (warp < kEtEpiWarps)
    et_epilogue<MODE, O>(a, groups, bars, units, tiles, ctiles, tmem, smem + (size_t)ring * stage_bytes, abort);
  else if (warp == kEtEpiWarps)
    loaded = et_loader<MODE>(a, groups, bars, base, stage_bytes, ring, units, tiles, ctiles, topk, abort);
  else
    issued = et_issuer<MODE>(a, groups, bars, base, stage_bytes, ring, units, tiles, ctiles, tmem, abort);
  tc_fence_before();
  __syncthreads();
  if (*abort) {  // (nobody sets it any more: the same for all)
    // what a CTA that gave up has in flight ends before its shared and tensor memory go
    int never = 0;
    for (int i = max(0, loaded - ring); i < loaded; ++i) mbar_wait_abort(&bars.full[i % ring], (i / ring) & 1, &never, kMxDrainNs);
    if (issued > 0) mbar_wait_abort(&bars.empty[(issued - 1) % ring], ((issued - 1) / ring) & 1, &never, kMxDrainNs);
    if (threadIdx.x == 0) atomicOr(a.flags, 2u);
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Boxes of 64 elements by `rows` rows (gathered: one). Box starts are multiples of 64 elements.
cudaError_t et_map(CUtensorMap* m, int dtype, const void* p, int cols, long rows, int64_t ld, int E, int64_t lde, int box) {
  const auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)E};
  cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(E > 1 ? lde : ld) * 2};
  cuuint32_t boxes[3] = {64, (cuuint32_t)box, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, dtype == TM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, E > 0 ? 3 : 2,
                         const_cast<void*>(p), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int MODE, typename O>
cudaError_t et_launch(const EtArgs& a, int topk, int sms, cudaStream_t st) {
  auto kern = k_ex_tc<MODE, O>;
  static OncePerDevice done;
  const cudaError_t limit = allow_smem(done, kern, (int)kEtSmem);
  if (limit != cudaSuccess) return limit;
  const uint32_t stage = kEtABytes + (uint32_t)a.bn * 128, store = MODE == kExGradW ? 0 : kEtEpiWarps / 4 * kEtStoreBytes;
  const int ring = (int)std::min<uint32_t>(kEtMaxRing, (kEtSmem - 1024 - store) / stage);
  const long tiles = (a.M + 127) / 128, ctiles = MODE == kExGradW ? (a.cols + a.bn - 1) / a.bn : 1;
  const long units = MODE == kExGradW ? (long)a.E * tiles * ctiles : ((long)a.R / a.bn + std::min<long>(a.R, a.E + 1)) * tiles;
  if (units >= 1L << 31) return cudaErrorInvalidConfiguration;
  const int grid = (int)std::max<long>(1, std::min<long>(units, sms));
  return launch_after(kern, dim3(grid), kEtThreads, 1024 + ring * stage + store, st, a, ring, FastDiv((uint32_t)tiles),
                      FastDiv((uint32_t)ctiles), FastDiv((uint32_t)topk));
}

bool et_rows_ok(const void* p, int64_t ld) { return ((uintptr_t)p) % 16 == 0 && ld % 8 == 0 && ld < (1LL << 38); }

}  // namespace

bool ex_tc_ok(const ExArgs& a) {
  if (a.T == 0) return false;
  if (a.mode != kExGradX && !et_rows_ok(a.x, a.ldx)) return false;
  if (a.mode != kExForward && !et_rows_ok(a.g, a.ldg)) return false;
  return a.mode == kExGradW || (et_rows_ok(a.w, a.ldw) && (a.E == 1 || (et_rows_ok(a.w, a.lde) && a.lde > 0)));
}

cudaError_t launch_ex_tc(const ExArgs& a, int sms, cudaStream_t st) {
  EtArgs t{};
  const int R = a.T * a.topk, es = a.out_dtype == TM_F32 ? 4 : 2;
  t.E = a.E, t.R = R, t.bf16 = a.dtype == TM_BF16, t.per_route = a.per_route;
  t.order = a.order, t.offsets = a.offsets, t.out = a.out, t.flags = a.flags;
  const long xrows = a.per_route ? R : a.T;
  cudaError_t e;
  if (a.mode == kExGradW) {
    t.M = a.N, t.cols = a.K, t.bn = std::min(256, (a.K + 63) / 64 * 64);
    e = et_map(&t.amap, a.dtype, a.g, a.N, R, a.ldg, 0, 0, 1);
    if (e == cudaSuccess) e = et_map(&t.bmap, a.dtype, a.x, a.K, xrows, a.ldx, 0, 0, 1);
    t.vec = ((uintptr_t)a.out) % 16 == 0 && (int64_t)a.K * es % 16 == 0;
  } else {
    const bool fwd = a.mode == kExForward;
    t.M = fwd ? a.N : a.K, t.depth = fwd ? a.K : a.N;
    // columns of a block: twice the mean number of routes of an expert, so that most experts
    // take one block and a stage holds no more than it needs (shorter stages: more in flight)
    t.bn = std::min(256, std::max(32, (2 * ((R + a.E - 1) / a.E) + 31) / 32 * 32));
    e = et_map(&t.amap, a.dtype, a.w, a.K, a.N, a.ldw, a.E, a.lde, fwd ? 128 : 64);
    if (e == cudaSuccess) e = fwd ? et_map(&t.bmap, a.dtype, a.x, a.K, xrows, a.ldx, 0, 0, 1)
                                  : et_map(&t.bmap, a.dtype, a.g, a.N, R, a.ldg, 0, 0, 1);
    t.vec = ((uintptr_t)a.out) % 16 == 0 && t.M % 8 == 0;
  }
  if (e != cudaSuccess) return e;
  auto go = [&](auto elem) {
    using O = decltype(elem);
    return a.mode == kExForward ? et_launch<kExForward, O>(t, a.topk, sms, st)
         : a.mode == kExGradX   ? et_launch<kExGradX, O>(t, a.topk, sms, st)
                                : et_launch<kExGradW, O>(t, a.topk, sms, st);
  };
  return TM_BY_DTYPE(a.out_dtype, go);
}

}  // namespace tmoe
