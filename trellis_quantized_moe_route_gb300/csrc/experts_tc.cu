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
// them, and results go straight to route order.
//
// Persistent, one CTA per SM: eight epilogue warps, sixteen that fetch rows, one for
// the weights, one that issues the MMAs.
//
// Measured on one GB300, us (floor: each operand once at the memory's copy rate):
//   160 experts 1536 -> 5120, 32768 routes   forward 466 to 476, dx 453 to 461, dW 640 to 655 (434 each). The
//     products run at the memory's rate but for a last round of units (5%). dW is bound by
//     what an SM exchanges with L2: for a tile of 256 x 256 and its 205 routes, 205 KB
//     come at 42 bytes a cycle (by TMA or cp.async or both) and 131 KB leave at 26
//     (also where dW stays in L2), some 5 us in all, and the two add up: half a tile
//     filled while the other half is drained takes 667. Tiles of 128 x 256 need half as many rows
//     again (876).
//   128 experts 1024 -> 1024, 16384 routes, uneven   62 to 66, 84 to 88 with the tokens' sums, 76 to 82 (45)
//   64 experts 2560 -> 640, 5120 routes   42 to 46, 64 to 67 with the sums, 50 to 53 (32)
//   8 tokens x 8 of 128 experts, 1024 -> 1024   19 to 23 (bytes 15)
//   (The first figure: ten calls in a CUDA graph.)
// Measured and not kept: dW's stages of 32 routes with two store buffers a warp (708 us;
// with 64 and room for two stages 742; two buffers of half the size 674), stores of dW from registers after exchanging
// pieces between four lanes (734), the routes of dW's stages looked up two stages
// ahead (656), forward's and dx's results stored from registers after such an exchange
// (501 and 469 us; through shared memory 480 and 462).
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
constexpr int kEtRowWarps = 16;
constexpr int kEtThreads = (kEtEpiWarps + kEtRowWarps + 2) * 32;
constexpr int kEtMaxRing = 12;
constexpr uint32_t kEtSmem = 227 * 1024;
constexpr uint32_t kEtABytes = 128 * 128;      // half a tile of A: 128 rows of 64 elements, or 64 of 128
constexpr uint32_t kEtGroup = 64 * 128;        // 64 rows of 64 elements (contiguous along M or N)
constexpr uint32_t kEtStoreBytes = 4096;       // results on their way: rows' for four epilogue warps, dW's for one
constexpr int kEtMaxGroups = 257 + 1;
constexpr int kEtHeights = 3;                  // that a tile of forward's weights may have: 128, 96 or 64 channels
constexpr int kEtBox = 32;                     // rows of its TMA copies

struct EtArgs {
  CUtensorMap map;          // forward, grad_x: the weights; grad_w: the result (if vec)
  CUtensorMap xmap, gmap;   // rows of x and dy, one at a time
  const uint16_t* x;
  int64_t ldx;              // elements
  int E, R, M, depth;       // M: output channels; depth: contraction (forward, grad_x)
  int cols;                 // grad_w: columns of dW
  int bn;                   // most columns of a unit
  int bufs;                 // accumulators of a tile that TMEM holds: 1 or 2
  int bf16, per_route, vec; // vec: results can be stored in 16-byte words
  const int32_t *order, *offsets;
  void* out;
  uint32_t* flags;
  uint64_t wait_ns;         // limit of a wait
  int stall;                // test of the bounded waits: which one never ends (kEtStall*, or 0)
};

struct EtBars {
  uint64_t full[kEtMaxRing], empty[kEtMaxRing];    // the ring of the rows
  uint64_t wfull[kEtMaxRing], wempty[kEtMaxRing];  // that of the weights
  uint64_t acc_full[2], acc_empty[2];
  uint64_t never;                                  // nothing arrives here
};

// Which wait runs out in a test: the issuer's before its first MMA, an epilogue warp's for every
// accumulator, that of the first or the last of the rows' warps before its first stage, the weights'.
enum { kEtStallIssuer = 1, kEtStallEpilogue, kEtStallFirstRows, kEtStallLastRows, kEtStallWeights };

// The groups of routes: where each begins; forward, grad_x: its first block; grad_w:
// the experts in the order in which they are taken.
struct EtGroups {
  int off[kEtMaxGroups], first[kEtMaxGroups];
  bool uneven;
};

// The CTA's unit of a round. grad_w's units last as long as their experts have routes:
// where that differs much, those with most routes come first, and rounds go to and
// fro, so that who has a long unit in one has a shorter one in the next (uneven: 90 -> 82
// us; large, where it hardly differs, would take 669 and not 660).
template <int MODE>
__device__ __forceinline__ int et_turn(const EtGroups& g, int round) {
  const int n = (int)gridDim.x;
  return round * n + (MODE == kExGradW && g.uneven && (round & 1) ? n - 1 - (int)blockIdx.x : (int)blockIdx.x);
}

// Two rings of stages of 64 of the contraction: the weights come from memory and
// need more of them in flight than the rows, which mostly come from L2. (One ring
// of both, 4 stages of 48 KB: 58% of the memory's rate at 205 routes an expert.)
// grad_w has both its operands in the rows' ring.
struct EtRings {
  int rows, weights;
  uint32_t stage;  // bytes of a stage of the rows' ring
};

// Channels of a tile, and tiles of that size.
struct EtTiles {
  int high;
  FastDiv tiles;
};

// Of forward's heights the one whose rounds of units take least. A unit's time
// goes by its weights; kEtUnit is what it takes besides, in channels. (320 units of
// 128 channels are three rounds on 152 SMs, 448 of 96 as well: odd 53 -> 46 us.)
constexpr int kEtUnit = 8;
struct EtChoice {
  EtTiles of[kEtHeights];
  __device__ __forceinline__ EtTiles pick(int blocks) const {
    EtTiles best = of[0];
    int least = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < kEtHeights; ++i) {
      const int units = blocks * (int)of[i].tiles.d, cost = (units + (int)gridDim.x - 1) / (int)gridDim.x * (of[i].high + kEtUnit);
      if (cost < least) least = cost, best = of[i];
    }
    return best;
  }
};

// What lies in shared memory behind the rings and the store buffers.
struct EtShared {
  EtBars bars;
  EtGroups groups;
  uint32_t tmem_slot;
  int abort;
};

struct EtUnit {
  int expert, tile, slot0, rows, depth;  // rows: columns of D; grad_w: tile of M, slot0 the first route, col0
  int col0;
};

// Halves of 128 channels of a unit's tile of MT * 128.
template <int MT>
__device__ __forceinline__ int et_halves(const EtArgs& a, const EtUnit& m) {
  return MT == 1 || a.M - m.tile * (MT * 128) > 128 ? MT : 1;
}

template <int MODE>
__device__ __forceinline__ EtUnit et_unit(const EtArgs& a, const EtGroups& g, int u, int units, FastDiv tiles, FastDiv ctiles) {
  EtUnit m;
  const int v = min(u, units - 1);
  int b = (int)tiles.div((uint32_t)v);
  m.tile = v - b * (int)tiles.d;
  if (MODE == kExGradW) {
    const int p = (int)ctiles.div((uint32_t)b);
    m.expert = g.first[p];
    m.col0 = (b - p * (int)ctiles.d) * a.bn;
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
template <int MODE, int MT>
__device__ int et_loader(const EtArgs& a, const EtGroups& g, EtBars& B, uint32_t base, int ring, int units, int high,
                         FastDiv tiles, FastDiv ctiles, volatile int* abort) {
  const bool lead = mx_elect();
  const uint32_t bar0 = smem_u32(&B.wfull[0]);
  if (a.stall == kEtStallWeights && !mx_wait_warp(&B.never, 0, abort, a.wait_ns)) return 0;
  MxRing r;
  int it = 0;
  for (int round = 0, u; (u = et_turn<MODE>(g, round)) < units; ++round) {
    const EtUnit m = et_unit<MODE>(a, g, u, units, tiles, ctiles);
    const int stages = (m.depth + 63) / 64, halves = et_halves<MT>(a, m), c0 = m.tile * high;
    for (int s = 0; s < stages; ++s, ++it, r.next(ring)) {
      if (it >= ring && !mx_wait_warp(&B.wempty[r.slot], r.phase ^ 1, abort, a.wait_ns)) return it;
      const uint32_t st = base + (uint32_t)r.slot * (MT * kEtABytes), bar = bar0 + (uint32_t)r.slot * 8;
      if (lead && MODE == kExForward && MT == 1) {
        mx_expect(bar, high * 128);
#pragma unroll
        for (int i = 0; i < 128; i += kEtBox)
          if (i < high) et_tma_3d(st + i * 128, &a.map, s * 64, c0 + i, m.expert, bar);
      } else if (lead) {
        mx_expect(bar, halves * kEtABytes);
#pragma unroll
        for (int h = 0; h < MT; ++h) {
          if (h >= halves) break;
          if (MODE == kExForward) {
            et_tma_3d(st + h * kEtABytes, &a.map, s * 64, c0 + h * 128, m.expert, bar);
          } else {
            et_tma_3d(st + h * kEtABytes, &a.map, c0 + h * 128, s * 64, m.expert, bar);
            et_tma_3d(st + h * kEtABytes + kEtGroup, &a.map, c0 + h * 128 + 64, s * 64, m.expert, bar);
          }
        }
      }
    }
  }
  return it;
}

// The rows' part of the stages, by sixteen warps: TMA copies of four rows (one warp
// alone took 65-73 cycles to issue each; sixteen together some 9 to 12), and for dW in
// tiles of 256 x's rows by cp.async, 16 bytes a lane (some 14 cycles for 512 of them).
// TMA and the load/store unit are different parts of the SM and together move
// more (large, dW: 745 us by TMA alone, 682 so; forward 478 by TMA, 489 and 526 with
// half and all of the rows by cp.async). cp.async writes by the generic proxy; the
// issuer's fence behind the stage's barrier shows it to the tensor cores.
template <int MODE, int MT>
struct EtRowPlan {
  static constexpr int kCopyWarps = MT == 2 && MODE == kExGradW ? 8 : 0;  // by cp.async: the last ones
  static constexpr int kTmaWarps = kEtRowWarps - kCopyWarps;
  static constexpr int kArrivals = kTmaWarps + 32 * kCopyWarps;  // of a stage
};

// What the row warps' walk through units and stages has in common. (Returns the
// stages.)
struct EtWalk {
  EtBars& B;
  volatile int* abort;
  uint64_t wait_ns;
  uint32_t base, stage_bytes;
  int ring, it;
  MxRing r;
  // waits for the stage's place; its shared address in `st`
  __device__ __forceinline__ bool next(uint32_t& st) {
    if (it >= ring && !mx_wait_warp(&B.empty[r.slot], r.phase ^ 1, abort, wait_ns)) return false;
    st = base + (uint32_t)r.slot * stage_bytes;
    return true;
  }
  __device__ __forceinline__ void done() {
    ++it;
    r.next(ring);
  }
};

// By TMA. (Returns the stages it loaded.)
template <int MODE, int MT>
__device__ int et_rows_tma(const EtArgs& a, const EtGroups& g, EtWalk k, int units, FastDiv tiles, FastDiv ctiles, FastDiv topk) {
  constexpr int kWarps = EtRowPlan<MODE, MT>::kTmaWarps;
  const int lane = threadIdx.x & 31, warp = (int)(threadIdx.x >> 5) - kEtEpiWarps;
  auto source = [&](int route) { return a.per_route ? route : (int)topk.div((uint32_t)route); };
  uint32_t st;
  for (int round = 0, u; (u = et_turn<MODE>(g, round)) < units; ++round) {
    const EtUnit m = et_unit<MODE>(a, g, u, units, tiles, ctiles);
    const int stages = (m.depth + 63) / 64;
    if constexpr (MODE == kExGradW) {
      // a lane for a group of 64 columns of four rows: first dy's groups, then (if it has no
      // warps of its own) x's; eight lanes to four rows
      constexpr int kQuads = 16 / kWarps;  // of a warp
      const int quad = warp * kQuads + (lane >> 3), c = lane & 7, c0 = m.tile * (MT * 128);
      const int agroups = min(2 * MT, (a.M - c0 + 63) / 64), groups = MT == 1 ? (m.rows + 63) / 64 : 0;
      int q[4];
      auto look = [&](int s) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = __ldg(a.order + m.slot0 + min(s * 64 + quad * 4 + i, m.depth - 1));
      };
      if (stages) look(0);
      for (int s = 0; s < stages; ++s, k.done()) {
        if (!k.next(st)) return k.it;
        const uint32_t bar = smem_u32(&k.B.full[k.r.slot]);
        const bool some = lane < 8 * kQuads && s * 64 + quad * 4 < (m.depth + 15) / 16 * 16;
        const bool isg = some && c < agroups, isx = MT == 1 && some && c < groups;
        const uint32_t bytes = 512u * (__popc(__ballot_sync(0xFFFFFFFFu, isg)) + __popc(__ballot_sync(0xFFFFFFFFu, isx)));
        if (lane == 0) mx_expect(bar, bytes);
        __syncwarp();
        if (isg) et_gather4(st + c * kEtGroup + quad * 512, &a.gmap, c0 + c * 64, q, bar);
        if (MT == 1) {
          __syncwarp();
          if (isx) {
            const int t[4] = {source(q[0]), source(q[1]), source(q[2]), source(q[3])};
            et_gather4(st + MT * kEtABytes + c * kEtGroup + quad * 512, &a.xmap, m.col0 + c * 64, t, bar);
          }
        }
        __syncwarp();
        if (s + 1 < stages) look(s + 1);
      }
    } else {
      // the first lanes of a warp: four rows each
      constexpr int kPer = 64 / kWarps;
      const int quad = warp + (lane % kPer) * kWarps, quads = et_up16(m.rows) / 4;
      int q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int route = __ldg(a.order + m.slot0 + min(quad * 4 + i, m.rows - 1));
        q[i] = MODE == kExForward ? source(route) : route;
      }
      const bool mine = lane < kPer && quad < quads;
      const uint32_t bytes = 512u * __popc(__ballot_sync(0xFFFFFFFFu, mine));
      for (int s = 0; s < stages; ++s, k.done()) {
        if (!k.next(st)) return k.it;
        const uint32_t bar = smem_u32(&k.B.full[k.r.slot]);
        if (lane == 0) mx_expect(bar, bytes);
        __syncwarp();
        if (mine) et_gather4(st + (uint32_t)quad * 512, MODE == kExForward ? &a.xmap : &a.gmap, s * 64, q, bar);
        __syncwarp();
      }
    }
  }
  return k.it;
}

// x's rows of dW's stages by cp.async; what it copied has landed when it returns.
template <int MODE, int MT>
__device__ void et_rows_copy(const EtArgs& a, const EtGroups& g, EtWalk k, int units, FastDiv tiles, FastDiv ctiles, FastDiv topk) {
  constexpr int kWarps = EtRowPlan<MODE, MT>::kCopyWarps, kSweep = kWarps * 4, kSweeps = 64 / kSweep;  // rows at once
  const int lane = threadIdx.x & 31, warp = (int)(threadIdx.x >> 5) - kEtEpiWarps - EtRowPlan<MODE, MT>::kTmaWarps;
  const int chunk = lane & 7, row = warp * 4 + (lane >> 3);
  const uint32_t at = (uint32_t)row * 128 + (uint32_t)((chunk ^ (row & 7)) << 4);
  uint32_t st;
  bool ok = true;
  for (int round = 0, u; ok && (u = et_turn<MODE>(g, round)) < units; ++round) {
    const EtUnit m = et_unit<MODE>(a, g, u, units, tiles, ctiles);
    const int stages = (m.depth + 63) / 64, k0 = m.col0 + chunk * 8, groups = (m.rows + 63) / 64;
    int route[kSweeps];
    auto look = [&](int s) {
#pragma unroll
      for (int h = 0; h < kSweeps; ++h) {
        const int i = s * 64 + h * kSweep + row;
        route[h] = i < m.depth ? __ldg(a.order + m.slot0 + i) : -1;
      }
    };
    if (stages) look(0);
    for (int s = 0; s < stages; ++s, k.done()) {
      if (!(ok = k.next(st))) break;
      const int rows = et_up16(min(64, m.depth - s * 64));
#pragma unroll
      for (int h = 0; h < kSweeps; ++h) {
        if (h * kSweep + row >= rows) break;
        const bool in = route[h] >= 0;  // (rows past the last route: zeros)
        const uint16_t* p = a.x + (in ? (size_t)(a.per_route ? route[h] : (int)topk.div((uint32_t)route[h])) * a.ldx + k0 : 0);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c >= groups) break;
          const int bytes = in ? min(16, max(0, (a.cols - k0 - c * 64) * 2)) : 0;
          et_copy(st + MT * kEtABytes + c * kEtGroup + h * kSweep * 128 + at, bytes ? p + c * 64 : a.x, bytes);
        }
      }
      cp_async_mbar_arrive(&k.B.full[k.r.slot]);
      if (s + 1 < stages) look(s + 1);
    }
  }
  asm volatile("cp.async.wait_all;\n" ::: "memory");
  __syncwarp();
}

// (returns the stages whose MMAs it issued)
template <int MODE, int MT>
__device__ int et_issuer(const EtArgs& a, const EtGroups& g, EtBars& B, uint32_t base, uint32_t wbase, EtRings rings, int units,
                         FastDiv tiles, FastDiv ctiles, uint32_t tmem, volatile int* abort) {
  const bool lead = mx_elect();
  if (a.stall == kEtStallIssuer && !mx_wait_warp(&B.never, 0, abort, a.wait_ns)) return 0;
  MxRing r, rw;
  int it = 0, nu = 0;
  for (int round = 0, u; (u = et_turn<MODE>(g, round)) < units; ++round) {
    const EtUnit m = et_unit<MODE>(a, g, u, units, tiles, ctiles);
    const int stages = (m.depth + 63) / 64;
    if (stages == 0) continue;
    const int buf = a.bufs == 2 ? nu & 1 : 0, turn = a.bufs == 2 ? nu >> 1 : nu;
    if (turn >= 1 && !mx_wait_warp(&B.acc_empty[buf], (turn - 1) & 1, abort, a.wait_ns)) return it;
    ++nu;
    tc_fence_after();
    const uint32_t idesc = et_idesc<MODE>(a.bf16, et_up16(m.rows)), d = tmem + (uint32_t)(buf * MT * a.bn);
    const int halves = et_halves<MT>(a, m);
    for (int s = 0; s < stages; ++s, ++it, r.next(rings.rows), rw.next(rings.weights)) {
      if (!mx_wait_warp(&B.full[r.slot], r.phase, abort, a.wait_ns)) return it;
      if (EtRowPlan<MODE, MT>::kCopyWarps) fence_proxy_async();
      if (MODE != kExGradW && !mx_wait_warp(&B.wfull[rw.slot], rw.phase, abort, a.wait_ns)) return it;
      const uint32_t st = base + (uint32_t)r.slot * rings.stage, wt = wbase + (uint32_t)rw.slot * (MT * kEtABytes);
      const int left = min(64, m.depth - s * 64), steps = (left + 15) / 16;
      if (MODE == kExGradW && (left & 15)) {
        // Rows past the last route, which the gather filled with some row, become zeros: of both
        // operands, since zero times infinity is none.
        const int groups = 2 * MT + (MT == 1 ? (m.rows + 63) / 64 : 0), lane = threadIdx.x & 31;
        for (int c = 0; c < groups; ++c)
          for (int i = left + (lane >> 3); i < et_up16(left); i += 4)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};\n" ::"r"(st + c * kEtGroup + i * 128 + (lane & 7) * 16), "r"(0)
                         : "memory");
        fence_proxy_async();
        __syncwarp();
      }
      tc_fence_after();
      const uint64_t ad = MODE == kExForward ? smem_desc_sw128(wt) : et_desc_mn(MODE == kExGradX ? wt : st);
      const uint64_t bd = MODE == kExGradW ? et_desc_mn(st + MT * kEtABytes) : smem_desc_sw128(st);
      constexpr uint64_t sa = MODE == kExForward ? 2 : 128, sb = MODE == kExGradW ? 128 : 2;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < steps) {
#pragma unroll
          for (int h = 0; h < MT; ++h)
            if (h < halves && lead)
              tc_mma_f16(d + (uint32_t)(h * a.bn), ad + (uint64_t)(h * (kEtABytes >> 4)) + k * sa, bd + k * sb, idesc,
                         s > 0 || k > 0 ? 1u : 0u);
        }
      if (lead) tc_commit(&B.empty[r.slot]);
      if (MODE != kExGradW && lead) tc_commit(&B.wempty[rw.slot]);
    }
    if (lead) tc_commit(&B.acc_full[buf]);
  }
  return it;
}

// 32 rows by 128 bytes of dW, a lane's row in v, by way of shared memory and one
// TMA store for the warp. (A lane's own 16-byte stores, each to its row, wrote dW at
// 2.6 TB/s.) What lies past the last row or column is left out by the copy.
__device__ __forceinline__ void et_store_tile(const uint4 (&v)[8], unsigned char* stage, const CUtensorMap* map, int x, int y, int z,
                                              bool on) {
  const int lane = threadIdx.x & 31;
  asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");  // (the lane that issued the last one: it has been read)
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) = v[c];
  fence_proxy_async();
  __syncwarp();
  if (lane == 0 && on) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n" ::"l"(map), "r"(x), "r"(y),
                 "r"(z), "r"(smem_u32(stage)) : "memory");
    asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
  }
}

// The same where dW's rows are not whole 16-byte words: element by element, lanes
// along a row; `rows` and `cols` of them are there.
template <typename O>
__device__ __forceinline__ void et_store_elements(const uint4 (&v)[8], unsigned char* stage, O* out, int ld, int rows, int cols) {
  constexpr int kCols = 128 / (int)sizeof(O);
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) = v[c];
  __syncwarp();
  const int n = min(rows, 32);
#pragma unroll 4
  for (int r = 0; r < n; ++r)
#pragma unroll
    for (int c = lane; c < kCols; c += 32) {
      const int b = c * (int)sizeof(O);
      if (c < cols) out[(size_t)r * ld + c] = *reinterpret_cast<const O*>(stage + r * 128 + ((((b >> 4) ^ (r & 7)) << 4) | (b & 15)));
    }
}

template <int MODE, int MT, typename O>
__device__ void et_epilogue(const EtArgs& a, const EtGroups& g, EtBars& B, int units, int high, FastDiv tiles, FastDiv ctiles,
                            uint32_t tmem, unsigned char* stage, volatile int* abort) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quarter = warp & 3, part = warp >> 2;
  const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
  O* out = static_cast<O*>(a.out);
  constexpr int kStep = kEtEpiWarps / 4 * 32, kPieces = 256 / kStep;  // a warp's pieces of 32 columns
  int nu = 0;
  for (int round = 0, u; (u = et_turn<MODE>(g, round)) < units; ++round) {
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
    const int buf = a.bufs == 2 ? nu & 1 : 0, turn = a.bufs == 2 ? nu >> 1 : nu, halves = et_halves<MT>(a, m);
    if (some) {
      const bool test = a.stall == kEtStallEpilogue && warp == 0;
      const bool full = mx_wait_warp(test ? &B.never : &B.acc_full[buf], test ? 0 : turn & 1, abort, a.wait_ns);
      // the warps of a part meet at its barrier while they store: they go on together or not at all
      if (!mx_vote_part(full, 1 + part)) break;
      ++nu;
      tc_fence_after();
    }
    // the accumulators are free when the warp's last piece of them is in registers
    bool held = some;
    auto release = [&]() {
      tc_fence_before();
      if (lane == 0) mbar_arrive(&B.acc_empty[buf]);
      __syncwarp();
      held = false;
    };
    for (int h = 0; h < halves; ++h) {
      const uint32_t d = tmem + lane_base + (uint32_t)((buf * MT + h) * a.bn);
      const int first = m.tile * high + h * 128, end = min(a.M, first + min(128, high)), n = first + quarter * 32 + lane;
      const bool last = h == halves - 1;
      if (MODE == kExGradW) {
        constexpr int kCols = 128 / (int)sizeof(O);  // columns of 128 bytes
        const int n0 = first + quarter * 32;
        for (int c0 = part * kCols; c0 < m.rows; c0 += kEtEpiWarps / 4 * kCols) {
          uint4 q[8];
          O* e = reinterpret_cast<O*>(q);
          if (some) {
#pragma unroll
            for (int i = 0; i < kCols; i += 32) {
              uint32_t v[32];
              tmem_ld32(d + c0 + i, v);
              tmem_ld_wait();
              reg_fence32(v);
#pragma unroll
              for (int c = 0; c < 32; ++c) e[i + c] = from_f32<O>(__uint_as_float(v[c]));
            }
            if (last && c0 + kEtEpiWarps / 4 * kCols >= m.rows) release();
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) q[c] = make_uint4(0, 0, 0, 0);
          }
          if (a.vec) {
            et_store_tile(q, stage + warp * kEtStoreBytes, &a.map, m.col0 + c0, n0, m.expert, n0 < a.M);
          } else {
            et_store_elements<O>(q, stage + warp * kEtStoreBytes, out + ((size_t)m.expert * a.M + n0) * a.cols + m.col0 + c0, a.cols,
                                 a.M - n0, m.rows - c0);
          }
          __syncwarp();  // (tcgen05.ld is for a converged warp)
        }
      }
#pragma unroll
      for (int k = 0; k < (MODE == kExGradW ? 0 : kPieces); ++k) {
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
          if (last && c0 + kStep >= m.rows) release();
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) y[c] = 0.0f;
        }
        if (sizeof(O) == 2 && a.vec)
          mx_store32_words<O>(y, out, row[k], m.rows - c0, first, end, a.M, stage + part * kEtStoreBytes, 1 + part);
        else
          mx_store32<O>(y, out, row[k], m.rows - c0, n < end ? n : a.M, a.M);
        __syncwarp();  // (tcgen05.ld is for a converged warp)
      }
    }
    if (held) release();  // (it had no piece)
  }
  if (MODE == kExGradW) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
}

template <int MODE>
constexpr uint32_t et_store_bytes() { return (MODE == kExGradW ? kEtEpiWarps : kEtEpiWarps / 4) * kEtStoreBytes; }

template <int MODE, int MT, typename O>
__global__ void __launch_bounds__(kEtThreads, 1) k_ex_tc(const __grid_constant__ EtArgs a, EtRings rings, EtChoice choice, FastDiv ctiles,
                                                         FastDiv topk) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t wofs = (uint32_t)rings.rows * rings.stage;
  unsigned char* store = smem + wofs + (uint32_t)rings.weights * (MT * kEtABytes);
  EtShared& sh = *reinterpret_cast<EtShared*>(store + et_store_bytes<MODE>());
  EtBars& bars = sh.bars;
  EtGroups& groups = sh.groups;
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < rings.rows; ++i) {
      mbar_init(&bars.full[i], EtRowPlan<MODE, MT>::kArrivals);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < rings.weights; ++i) {
      mbar_init(&bars.wfull[i], 1);
      mbar_init(&bars.wempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], kEtEpiWarps);
    }
    mbar_init(&bars.never, 1);
    sh.abort = 0;
    mbar_fence_init();
  }
  if (MODE != kExGradW && threadIdx.x == kEtEpiWarps * 32) mx_prefetch_map(&a.map);
  __syncwarp();
  if (warp == 0) tmem_alloc(&sh.tmem_slot, 512);
  grid_wait();
  grid_launch();
  for (int e = threadIdx.x; e <= a.E; e += kEtThreads) groups.off[e] = a.offsets[e];
  if (threadIdx.x == 0) groups.off[a.E + 1] = a.R;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (MODE == kExGradW) {
    int count[8], most = 0;  // of experts lane + 32 i
#pragma unroll
    for (int i = 0; i < 8; ++i) count[i] = lane + 32 * i < a.E ? groups.off[lane + 32 * i + 1] - groups.off[lane + 32 * i] : -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, count[i]);
    const bool uneven = __reduce_max_sync(0xFFFFFFFFu, most) > 2 * (a.R / a.E) + 64;  // (64: a stage)
    if (threadIdx.x == 0) groups.uneven = uneven;
    for (int e = warp; e < a.E; e += kEtThreads / 32) {
      const int n = groups.off[e + 1] - groups.off[e];
      int before = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) before += count[i] > n || (count[i] == n && lane + 32 * i < e);
      before = __reduce_add_sync(0xFFFFFFFFu, before);
      if (lane == 0) groups.first[uneven ? before : e] = e;
    }
  }
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
  const uint32_t tmem = sh.tmem_slot, base = smem_u32(smem);
  const EtTiles shape = MODE == kExForward && MT == 1 ? choice.pick(groups.first[a.E + 1]) : choice.of[0];
  const FastDiv tiles = shape.tiles;
  const int units = MODE == kExGradW ? a.E * (int)ctiles.d * (int)tiles.d : groups.first[a.E + 1] * (int)tiles.d;
  volatile int* abort = &sh.abort;
  int loaded = 0, rows_loaded = 0, issued = 0;
  if (warp < kEtEpiWarps)
    et_epilogue<MODE, MT, O>(a, groups, bars, units, shape.high, tiles, ctiles, tmem, store, abort);
  else if (warp < kEtEpiWarps + kEtRowWarps) {
    const EtWalk walk{bars, abort, a.wait_ns, base, rings.stage, rings.rows, 0, MxRing()};
    using Plan = EtRowPlan<MODE, MT>;
    const bool test = (a.stall == kEtStallFirstRows && warp == kEtEpiWarps) ||
                      (a.stall == kEtStallLastRows && warp == kEtEpiWarps + kEtRowWarps - 1);
    if (!test || mx_wait_warp(&bars.never, 0, abort, a.wait_ns)) {
      if (warp < kEtEpiWarps + Plan::kTmaWarps) rows_loaded = et_rows_tma<MODE, MT>(a, groups, walk, units, tiles, ctiles, topk);
      if constexpr (Plan::kCopyWarps > 0)
        if (warp >= kEtEpiWarps + Plan::kTmaWarps) et_rows_copy<MODE, MT>(a, groups, walk, units, tiles, ctiles, topk);
    }
  } else if (warp == kEtEpiWarps + kEtRowWarps) {
    if (MODE != kExGradW) loaded = et_loader<MODE, MT>(a, groups, bars, base + wofs, rings.weights, units, shape.high, tiles, ctiles, abort);
  } else
    issued = et_issuer<MODE, MT>(a, groups, bars, base, base + wofs, rings, units, tiles, ctiles, tmem, abort);
  tc_fence_before();
  __syncthreads();
  if (*abort) {  // (nobody sets it any more: the same for all)
    // What a CTA that gave up has in flight ends before its shared and tensor memory go. (A
    // stage that some warps never filled is waited for until the limit, by when the others'
    // copies have landed; cp.async's have been waited for.)
    int never = 0;
    for (int i = max(0, loaded - rings.weights); i < loaded; ++i)
      mbar_wait_abort(&bars.wfull[i % rings.weights], (i / rings.weights) & 1, &never, kMxDrainNs);
    for (int i = max(0, rows_loaded - rings.rows); i < rows_loaded; ++i)
      mbar_wait_abort(&bars.full[i % rings.rows], (i / rings.rows) & 1, &never, kMxDrainNs);
    if (issued > 0) mbar_wait_abort(&bars.empty[(issued - 1) % rings.rows], ((issued - 1) / rings.rows) & 1, &never, kMxDrainNs);
    if (threadIdx.x == 0) atomicOr(a.flags, 2u);
    __syncthreads();
  }
  tc_fence_after();
  __syncwarp();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// [E, N, K] in boxes of `width` elements (128 bytes, as all box starts are multiples of) by `box` rows.
cudaError_t et_map3(CUtensorMap* m, int dtype, const void* p, const ExArgs& a, int64_t ldw, int64_t lde, int width, int box) {
  const cuuint64_t dims[3] = {(cuuint64_t)a.K, (cuuint64_t)a.N, (cuuint64_t)a.E};
  const cuuint64_t es = dtype_bytes(dtype);
  const cuuint64_t strides[2] = {(cuuint64_t)ldw * es, (cuuint64_t)(a.E > 1 ? lde : ldw) * es};
  const cuuint32_t boxes[3] = {(cuuint32_t)width, (cuuint32_t)box, 1};
  return tensor_map_encode(m,
                           dtype == TM_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                           : dtype == TM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                           3, p, dims, strides, boxes);
}

cudaError_t et_map2(CUtensorMap* m, int dtype, const void* p, int cols, long rows, int64_t ld) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t boxes[2] = {64, 1};
  return tensor_map_encode(m, dtype == TM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, p, dims,
                           strides, boxes);
}

template <int MODE, int MT, typename O>
cudaError_t et_launch(EtArgs a, int topk, int sms, cudaStream_t st) {
  auto kern = k_ex_tc<MODE, MT, O>;
  static OncePerDevice done;
  const cudaError_t limit = allow_smem(done, kern, (int)kEtSmem);
  if (limit != cudaSuccess) return limit;
  const uint32_t rest = et_store_bytes<MODE>() + (uint32_t)sizeof(EtShared), room = kEtSmem - rest;
  EtRings rings;
  if (MODE == kExGradW) {
    rings.stage = MT * kEtABytes + (uint32_t)a.bn * 128;
    rings.rows = (int)std::min<uint32_t>(kEtMaxRing, room / rings.stage);
    rings.weights = 0;
  } else {
    rings.stage = (uint32_t)a.bn * 128;
    rings.rows = (int)std::min<uint32_t>(8, 96 * 1024 / rings.stage);  // (3 of 256 rows)
    rings.weights = (int)std::min<uint32_t>(kEtMaxRing, (room - rings.rows * rings.stage) / (MT * kEtABytes));
  }
  a.bufs = 2 * MT * a.bn <= 512 ? 2 : 1;
  auto of = [&](int high) { return EtTiles{high, FastDiv((uint32_t)((a.M + high - 1) / high))}; };
  constexpr bool kChoose = MODE == kExForward && MT == 1;
  const EtChoice choice{{of(MT * 128), of(kChoose ? 96 : MT * 128), of(kChoose ? 64 : MT * 128)}};
  const long tiles = choice.of[2].tiles.d, ctiles = MODE == kExGradW ? (a.cols + a.bn - 1) / a.bn : 1;
  const long units = MODE == kExGradW ? (long)a.E * tiles * ctiles : ((long)a.R / a.bn + std::min<long>(a.R, a.E + 1)) * tiles;
  if (units >= 1L << 31) return cudaErrorInvalidConfiguration;
  const int grid = (int)std::max<long>(1, std::min<long>(units, sms));
  return launch_after(kern, dim3(grid), kEtThreads, rings.rows * rings.stage + rings.weights * (MT * kEtABytes) + rest, st, a, rings, choice,
                      FastDiv((uint32_t)ctiles), FastDiv((uint32_t)topk));
}

// Whether tiles have 256 channels, not 128: then the rows, which every tile of
// channels reads anew, are read half as often, and where there are many of them
// to an expert that counts (large: 205 routes an expert, forward 568 -> 480 us, dx 592
// -> 462, dW 840 -> 745; uneven: 128, 74 -> 66, 99 -> 89, 103 -> 96). With few, the
// weights are all that counts, and more, smaller tiles spread better over the SMs
// (one token: dx 27.1 us with 128 and 31.4 with 256; decode: 23.1 and 23.9; odd, 80
// routes an expert: 52.7 and 52.1, 67.3 and 66.7, dW 55.5 and 59.7).
bool et_wide(int R, int E) { return R >= 96L * E; }

}  // namespace

cudaError_t launch_ex_tc(const ExArgs& a, int sms, cudaStream_t st) {
  EtArgs t{};
  const int R = a.T * a.topk, es = a.out_dtype == TM_F32 ? 4 : 2;
  bool wide = et_wide(R, a.E);
  // Smaller units, as long as twice as many still find an SM each (433 routes of 3 experts,
  // 2560 -> 384: forward 32.9 -> 15.6 us; 3094 of 7, 256 -> 128: dW 14.8 -> 10.8).
  // `blocks`: about how many there are of bn columns.
  auto spread = [&](int M, auto blocks, int least) {
    while ((long)blocks(t.bn) * ((M + (wide ? 255 : 127)) / (wide ? 256 : 128)) * 2 <= sms) {
      if (wide)
        wide = false;
      else if (t.bn > least)
        t.bn = std::max(least, (t.bn / 2 + least - 1) / least * least);
      else
        break;
    }
  };
  t.E = a.E, t.R = R, t.bf16 = a.dtype == TM_BF16, t.per_route = a.per_route;
  t.order = a.order, t.offsets = a.offsets, t.out = a.out, t.flags = a.flags;
  t.wait_ns = a.wait_ns ? a.wait_ns : kMxWaitNs, t.stall = a.stall;
  t.x = static_cast<const uint16_t*>(a.x), t.ldx = a.ldx;
  if (a.mode != kExGradX) {
    const cudaError_t e = et_map2(&t.xmap, a.dtype, a.x, a.K, a.per_route ? R : a.T, a.ldx);
    if (e != cudaSuccess) return e;
  }
  if (a.mode != kExForward) {
    const cudaError_t e = et_map2(&t.gmap, a.dtype, a.g, a.N, R, a.ldg);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = cudaSuccess;
  if (a.mode == kExGradW) {
    t.M = a.N, t.cols = a.K, t.bn = std::min(256, (a.K + 63) / 64 * 64);
    spread(t.M, [&](int bn) { return std::min(R, a.E) * ((a.K + bn - 1) / bn); }, 64);
    t.vec = ((uintptr_t)a.out) % 16 == 0 && (int64_t)a.K * es % 16 == 0;
    if (t.vec) e = et_map3(&t.map, a.out_dtype, a.out, a, a.K, (int64_t)a.N * a.K, 128 / es, 32);
  } else {
    const bool fwd = a.mode == kExForward;
    t.M = fwd ? a.N : a.K, t.depth = fwd ? a.K : a.N;
    // columns of a block: twice the mean number of routes of an expert, so that most experts
    // take one block and a stage holds no more than it needs (shorter stages: more in flight)
    t.bn = std::min(256, std::max(32, (2 * ((R + a.E - 1) / a.E) + 31) / 32 * 32));
    spread(t.M, [&](int bn) { return std::max((R + bn - 1) / bn, std::min(R, a.E)); }, 32);
    e = et_map3(&t.map, a.dtype, a.w, a, a.ldw, a.lde, 64, !fwd ? 64 : wide ? 128 : kEtBox);
    t.vec = ((uintptr_t)a.out) % 16 == 0 && t.M % 8 == 0;
  }
  if (e != cudaSuccess) return e;
  auto go = [&](auto elem) {
    using O = decltype(elem);
    if (a.mode == kExForward)
      return wide ? et_launch<kExForward, 2, O>(t, a.topk, sms, st) : et_launch<kExForward, 1, O>(t, a.topk, sms, st);
    if (a.mode == kExGradX)
      return wide ? et_launch<kExGradX, 2, O>(t, a.topk, sms, st) : et_launch<kExGradX, 1, O>(t, a.topk, sms, st);
    return wide ? et_launch<kExGradW, 2, O>(t, a.topk, sms, st) : et_launch<kExGradW, 1, O>(t, a.topk, sms, st);
  };
  return TM_BY_DTYPE(a.out_dtype, go);
}

}  // namespace tmoe
