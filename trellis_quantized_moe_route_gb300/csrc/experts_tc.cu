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
// these products by their bytes, are read by every block once. Rows of x and dy
// are fetched where they lie, by the plan's order: there is no sorted copy of
// them, and results go straight to route order. Eight warps fetch them (16 bytes
// a lane, written in the swizzled layout); the weights come by TMA. (TMA's gather
// of four rows, issued lane by lane, took 65-73 cycles each: 1.8 us for a stage
// of 208 rows, of which the MMAs need 0.2.)
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
constexpr int kEtRowWarps = 8;
constexpr int kEtThreads = (kEtEpiWarps + kEtRowWarps + 2) * 32;
constexpr int kEtMaxRing = 12;
constexpr uint32_t kEtSmem = 224 * 1024;
constexpr uint32_t kEtABytes = 128 * 128;      // 128 rows of 64 elements, or 64 of 128
constexpr uint32_t kEtGroup = 64 * 128;        // 64 rows of 64 elements (contiguous along M or N)
constexpr uint32_t kEtStoreBytes = 16 * 256;   // for four epilogue warps
constexpr int kEtMaxGroups = 257 + 1;

struct EtArgs {
  CUtensorMap wmap;         // forward, grad_x
  const void *x, *g;
  int64_t ldx, ldg;         // elements
  int E, R, M, depth;       // M: output channels; depth: contraction (forward, grad_x)
  int cols;                 // grad_w: columns of dW
  int bn;                   // most columns of a unit
  int bf16, per_route, vec; // vec: results can be stored in 16-byte words
  const int32_t *order, *offsets;
  void* out;
  uint32_t* flags;
};

struct EtBars {
  uint64_t full[kEtMaxRing], wfull[kEtMaxRing];  // the rows' part of a stage, the weights' part
  uint64_t empty[kEtMaxRing];
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
// 16 bytes to shared memory, of which the last 16 - `bytes` are zeros.
__device__ __forceinline__ void et_copy(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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

// The weights' part of the stages. (Returns the stages it loaded.)
template <int MODE>
__device__ int et_loader(const EtArgs& a, const EtGroups& g, EtBars& B, uint32_t base, uint32_t stage_bytes, int ring, int units,
                         FastDiv tiles, FastDiv ctiles, volatile int* abort) {
  const bool lead = mx_elect();
  const uint32_t bar0 = smem_u32(&B.wfull[0]);
  MxRing r;
  int it = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const EtUnit m = et_unit<MODE>(a, g, u, units, tiles, ctiles);
    const int stages = (m.depth + 63) / 64;
    for (int s = 0; s < stages; ++s, ++it, r.next(ring)) {
      if (it >= ring && !mx_wait_warp(&B.empty[r.slot], r.phase ^ 1, abort, kMxWaitNs)) return it;
      const uint32_t st = base + (uint32_t)r.slot * stage_bytes, bar = bar0 + (uint32_t)r.slot * 8;
      if (lead) {
        mx_expect(bar, kEtABytes);
        if (MODE == kExForward) {
          et_tma_3d(st, &a.wmap, s * 64, m.tile * 128, m.expert, bar);
        } else {
          et_tma_3d(st, &a.wmap, m.tile * 128, s * 64, m.expert, bar);
          et_tma_3d(st + kEtGroup, &a.wmap, m.tile * 128 + 64, s * 64, m.expert, bar);
        }
      }
    }
  }
  return it;
}

// The rows' part. A lane copies 16 bytes of every 32nd row, and arrives at the
// stage's barrier when they have landed. (They are written by the generic proxy;
// the issuer's fence, behind that barrier, shows them to the tensor cores.)
template <int MODE>
__device__ void et_rows(const EtArgs& a, const EtGroups& g, EtBars& B, uint32_t base, uint32_t stage_bytes, int ring, int units,
                        FastDiv tiles, FastDiv ctiles, FastDiv topk, volatile int* abort) {
  const int lane = threadIdx.x & 31, warp = (int)(threadIdx.x >> 5) - kEtEpiWarps;
  const int chunk = lane & 7, row = warp * 4 + (lane >> 3);  // of each 32 rows
  const uint32_t at = (uint32_t)row * 128 + (uint32_t)((chunk ^ (row & 7)) << 4);
  const uint16_t *x = static_cast<const uint16_t*>(a.x), *dy = static_cast<const uint16_t*>(a.g);
  auto source = [&](int route) { return a.per_route ? route : (int)topk.div((uint32_t)route); };
  MxRing r;
  int it = 0;
  auto stage = [&](auto copy) {  // one stage's copies
    if (it >= ring && !mx_wait_warp(&B.empty[r.slot], r.phase ^ 1, abort, kMxWaitNs)) return false;
    copy(base + (uint32_t)r.slot * stage_bytes + at);
    cp_async_mbar_arrive(&B.full[r.slot]);
    ++it;
    r.next(ring);
    return true;
  };
  bool ok = true;
  if (MODE == kExGradW) {
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const EtUnit m = et_unit<MODE>(a, g, u, units, tiles, ctiles);
      const int stages = (m.depth + 63) / 64, groups = (m.rows + 63) / 64;
      int route[2];
      auto routes = [&](int s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = s * 64 + h * 32 + row;
          route[h] = i < m.depth ? __ldg(a.order + m.slot0 + i) : -1;
        }
      };
      if (stages) routes(0);
      const int n0 = m.tile * 128 + chunk * 8, k0 = m.col0 + chunk * 8;
      for (int s = 0; s < stages && ok; ++s) {
        ok = stage([&](uint32_t to) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h * 32 >= et_up16(m.depth - s * 64)) break;
            const bool in = route[h] >= 0;  // (rows past the last route: zeros)
            const uint16_t* p = dy + (in ? (size_t)route[h] * a.ldg : 0);
            const uint16_t* q = x + (in ? (size_t)source(route[h]) * a.ldx : 0);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int bytes = in ? min(16, max(0, (a.M - n0 - c * 64) * 2)) : 0;
              et_copy(to + c * kEtGroup + h * 4096, bytes ? p + n0 + c * 64 : dy, bytes);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (c >= groups) break;
              const int bytes = in ? min(16, max(0, (a.cols - k0 - c * 64) * 2)) : 0;
              et_copy(to + kEtABytes + c * kEtGroup + h * 4096, bytes ? q + k0 + c * 64 : x, bytes);
            }
          }
        });
        if (s + 1 < stages) routes(s + 1);
      }
    }
  } else {
    const uint16_t* src = MODE == kExForward ? x : dy;
    const int64_t ld = MODE == kExForward ? a.ldx : a.ldg;
    // a unit's rows are looked up while the one before it is copied
    auto find = [&](int u, int (&to)[8], EtUnit& m) {
      m = et_unit<MODE>(a, g, u, units, tiles, ctiles);
#pragma unroll
      for (int j = 0; j < 8; ++j)  // (past the last row: any)
        to[j] = j * 32 < m.rows ? __ldg(a.order + m.slot0 + min(j * 32 + row, m.rows - 1)) : 0;
    };
    int next[8];
    EtUnit m, ahead;
    if ((int)blockIdx.x < units) find(blockIdx.x, next, ahead);
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      m = ahead;
      const uint16_t* p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = src + (size_t)(MODE == kExForward ? source(next[j]) : next[j]) * ld + chunk * 8;
      if (u + (int)gridDim.x < units) find(u + gridDim.x, next, ahead);
      const int stages = (m.depth + 63) / 64, rows = et_up16(m.rows);
      for (int s = 0; s < stages && ok; ++s) {
        const int left = (m.depth - s * 64 - chunk * 8) * 2, bytes = min(16, max(0, left));
        ok = stage([&](uint32_t to) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j * 32 + row < rows) et_copy(to + kEtABytes + j * 4096, bytes ? p[j] + s * 64 : src, bytes);
        });
      }
    }
  }
  asm volatile("cp.async.wait_all;\n" ::: "memory");
}

// (returns the stages whose MMAs it issued)
template <int MODE>
__device__ int et_issuer(const EtArgs& a, const EtGroups& g, EtBars& B, uint32_t base, uint32_t stage_bytes, int ring, int units,
                         FastDiv tiles, FastDiv ctiles, uint32_t tmem, volatile int* abort) {
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
      if (MODE != kExGradW && !mx_wait_warp(&B.wfull[r.slot], r.phase, abort, kMxWaitNs)) return it;
      if (!mx_wait_warp(&B.full[r.slot], r.phase, abort, kMxWaitNs)) return it;
      fence_proxy_async();
      const uint32_t st = base + (uint32_t)r.slot * stage_bytes;
      const int steps = (min(64, m.depth - s * 64) + 15) / 16;
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
  constexpr int kStep = kEtEpiWarps / 4 * 32, kPieces = 256 / kStep;  // a warp's pieces of 32 columns
  int nu = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const EtUnit m = et_unit<MODE>(a, g, u, units, tiles, ctiles);
    int row[kPieces] = {};
    if (MODE != kExGradW) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int c = part * 32 + k * kStep + lane;
        row[k] = c < m.rows ? __ldg(a.order + m.slot0 + c) : 0;
      }
    }
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
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int c0 = part * 32 + k * kStep;
      if (c0 >= m.rows) break;
      float y[32];
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
        mx_store32_words<O>(y, out, row[k], m.rows - c0, m.tile, a.M, stage + part * kEtStoreBytes, 1 + part);
      } else {
        mx_store32<O>(y, out, row[k], m.rows - c0, n, a.M);
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
      mbar_init(&bars.full[i], kEtRowWarps * 32);
      mbar_init(&bars.wfull[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], kEtEpiWarps);
    }
    s_abort = 0;
    mbar_fence_init();
  }
  if (MODE != kExGradW && threadIdx.x == kEtEpiWarps * 32) mx_prefetch_map(&a.wmap);
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
  else if (warp < kEtEpiWarps + kEtRowWarps)
    et_rows<MODE>(a, groups, bars, base, stage_bytes, ring, units, tiles, ctiles, topk, abort);
  else if (warp == kEtEpiWarps + kEtRowWarps) {
    if (MODE != kExGradW) loaded = et_loader<MODE>(a, groups, bars, base, stage_bytes, ring, units, tiles, ctiles, abort);
  } else
    issued = et_issuer<MODE>(a, groups, bars, base, stage_bytes, ring, units, tiles, ctiles, tmem, abort);
  tc_fence_before();
  __syncthreads();
  if (*abort) {  // (nobody sets it any more: the same for all)
    // what a CTA that gave up has in flight ends before its shared and tensor memory go (the
    // row warps have waited for their copies)
    int never = 0;
    for (int i = max(0, loaded - ring); i < loaded; ++i) mbar_wait_abort(&bars.wfull[i % ring], (i / ring) & 1, &never, kMxDrainNs);
    if (issued > 0) mbar_wait_abort(&bars.empty[(issued - 1) % ring], ((issued - 1) / ring) & 1, &never, kMxDrainNs);
    if (threadIdx.x == 0) atomicOr(a.flags, 2u);
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Boxes of 64 elements by `box` rows. Box starts are multiples of 64 elements.
cudaError_t et_weight_map(CUtensorMap* m, const ExArgs& a, int box) {
  const auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[3] = {(cuuint64_t)a.K, (cuuint64_t)a.N, (cuuint64_t)a.E};
  cuuint64_t strides[2] = {(cuuint64_t)a.ldw * 2, (cuuint64_t)(a.E > 1 ? a.lde : a.ldw) * 2};
  cuuint32_t boxes[3] = {64, (cuuint32_t)box, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, a.dtype == TM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                         const_cast<void*>(a.w), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
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
  t.x = a.x, t.ldx = a.ldx, t.g = a.g, t.ldg = a.ldg;
  cudaError_t e = cudaSuccess;
  if (a.mode == kExGradW) {
    t.M = a.N, t.cols = a.K, t.bn = std::min(256, (a.K + 63) / 64 * 64);
    t.vec = ((uintptr_t)a.out) % 16 == 0 && (int64_t)a.K * es % 16 == 0;
  } else {
    const bool fwd = a.mode == kExForward;
    t.M = fwd ? a.N : a.K, t.depth = fwd ? a.K : a.N;
    // columns of a block: twice the mean number of routes of an expert, so that most experts
    // take one block and a stage holds no more than it needs (shorter stages: more in flight)
    t.bn = std::min(256, std::max(32, (2 * ((R + a.E - 1) / a.E) + 31) / 32 * 32));
    e = et_weight_map(&t.wmap, a, fwd ? 128 : 64);
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
