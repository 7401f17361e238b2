// Products with MXFP4 weights on the tensor cores (sm_103a).
//
// D[n, r] = sum_k W[n, k] x[r, k], both operands E2M1 codes with one E8M0 scale
// per 32 columns, as `tcgen05.mma.kind::mxf4.block_scale`: the 128 rows of a
// tile of W are the M side (TMEM lanes), the rows of x the N side (TMEM
// columns), so that a block of x may have any multiple of 16 rows up to 240
// and an expert with few routes wastes little. A thread of the epilogue then
// holds one output channel. Gated products keep two accumulators, gate and up
// rows of the same 128 channels against one x operand, and the same thread
// holds both.
//
// Persistent, one CTA per SM: a loader warp (TMA boxes of 256 columns = one
// 128-byte swizzle span of codes, bulk copies of the scale chunks), an issuer
// warp (scales to tensor memory with tcgen05.cp, then one MMA per 64
// columns), and sixteen epilogue warps that drain one accumulator buffer while
// the next unit fills the other. 240 columns twice, plus 24 columns of scales,
// is what 512 columns of tensor memory hold; that is why a block ends at 240
// (gated: 4 x 112).
//
// Measured on one GB300 (bf16 in and out, with quantisation and map, replayed from
// a CUDA graph; a call through the Python binding takes 1-5 us more where the
// host is the longer side):
//   2048 x 4096 x 4096 dense        20 us   3.4 PFLOP/s over the call. The
//     issuer spends 503 cycles on a stage of four 128 x 240 x 64 MMAs: 96 waiting
//     for data, 257 on the scales' copies and the MMAs, 26 on the commit and 124 in
//     its loop; the tensor pipe is active in 35% of the kernel's cycles. While an
//     epilogue reads the other buffer a stage takes 1100. Quantisation and
//     launches are 7 us of the call, the pipeline's start and last drain 3 us.
//   2048 tokens x 8 of 128 experts, gated 1024 -> 512, Zipf   26 us: map and
//     quantisation 7 us, then 49 KB a stage at 55-65 bytes a cycle and SM from
//     L2 and an epilogue of the same length (silu: two special-function
//     instructions a value).
//   4096 tokens x 8 of 160 experts, 1536 -> 5120   189.5 us: 1.03 GB of weights and
//     results in 155 us = 6.6 TB/s in the products, at the memory's rate.
// Timing copies without the MMAs, the stores or the loads each take as long or
// 2-3 us less in the first two: the three overlap.
//
// Every wait is bounded (2 s): one that runs out raises bit 1 of the error
// word, lets the copies and MMAs in flight finish, frees the tensor memory and
// returns.
#include <algorithm>

#include "elem.cuh"
#include "mxfp4.cuh"
#include "mxfp4.h"
#include "mxfp4_mma.cuh"
#include "status.h"
#include "tensor_map.h"
#include "tile_store.cuh"

namespace tmoe {

namespace {

constexpr int kMxEpiWarps = 16;
constexpr int kMxThreads = (kMxEpiWarps + 2) * 32;
constexpr int kMxMaxStages = 8;
constexpr int kMxSfCol = 480;       // first tensor-memory column of the scales
constexpr uint32_t kMxSmem = 226 * 1024;
constexpr int kMxStoreBytes = 16 * 256;  // 16 rows of 128 16-bit channels, for each four epilogue warps

struct MxBars {
  uint64_t full[kMxMaxStages], empty[kMxMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t never;  // nothing arrives on it (test of the bounded waits)
};

// One unit: a block of rows times 128 output channels.
struct MxUnit {
  int expert, tile, slot0, rows;
};

// Unit u (past the last one: the last, whose values are not used). Without a
// branch, so that a unit can be read ahead: the load is waited for where its
// values are used.
template <bool EXPERTS>
__device__ __forceinline__ MxUnit mx_unit(const MxTcArgs& a, int u, int units, FastDiv tiles) {
  MxUnit m;
  const int v = min(u, units - 1), b = (int)tiles.div((uint32_t)v);
  m.tile = v - b * (int)tiles.d;
  m.slot0 = b * a.bn;
  if (EXPERTS) {
    const int2 i = __ldg(a.block_info + b);  // (the map's, complete before this kernel starts)
    m.expert = i.x;
    m.rows = i.y;
  } else {
    m.expert = 0;
    m.rows = min(a.bn, a.rows - m.slot0);
  }
  return m;
}

struct MxGeom {
  FastDiv tiles;
  int units, stages, ring, ksteps;
  uint32_t a_bytes, b_bytes, sfa_bytes, sfb_bytes, stage_bytes;
};

template <bool GATED, bool EXPERTS>
__device__ __forceinline__ MxGeom mx_geom(const MxTcArgs& a, int ring, FastDiv tiles) {
  MxGeom g{tiles};
  const int blocks = EXPERTS ? *a.nblocks : (a.rows + a.bn - 1) / a.bn;
  g.units = blocks * (int)tiles.d;
  g.stages = mx_stages(a.K);
  g.ksteps = (mx_blocks(a.K) + 1) / 2;
  g.ring = ring;
  g.a_bytes = (GATED ? 2 : 1) * kMxTileBytes;
  g.b_bytes = (uint32_t)a.bn * 128;
  g.sfa_bytes = (GATED ? 2 : 1) * 1024;
  g.sfb_bytes = (uint32_t)a.nrb * 1024;
  g.stage_bytes = (g.a_bytes + g.b_bytes + g.sfa_bytes + g.sfb_bytes + 1023) / 1024 * 1024;
  return g;
}

// (returns the stages it loaded)
template <bool GATED, bool EXPERTS>
__device__ int mx_loader(const MxTcArgs& a, const MxGeom& g, MxBars& B, unsigned char* smem, volatile int* abort,
                         uint64_t limit) {
  const bool lead = mx_elect();
  const uint32_t base = smem_u32(smem), bar0 = smem_u32(&B.full[0]);
  const uint32_t bytes = g.a_bytes + g.b_bytes + g.sfa_bytes + g.sfb_bytes;
  // W's part of a stage: the copies of the codes and scales
  auto load_w = [&](int s, uint32_t st, uint32_t bar, int wrow, const uint8_t* wsf, const uint8_t* usf) {
    const uint32_t sf = st + g.a_bytes + g.b_bytes;
    if (lead) {
      mx_expect(bar, bytes);
      mx_tma_2d(st, &a.wmap, s * 128, wrow, bar);
      if (GATED) mx_tma_2d(st + kMxTileBytes, &a.wmap, s * 128, wrow + a.N, bar);
      mx_bulk(sf, wsf + s * 1024, 1024, bar);
      if (GATED) mx_bulk(sf + 1024, usf + s * 1024, 1024, bar);
    }
  };
  MxRing r;
  int it = 0, ahead = 0;
  bool ok = true;
  MxUnit next = mx_unit<EXPERTS>(a, blockIdx.x, g.units, g.tiles);
  {
    // The kernel before this one quantises x, and lets this one start only after
    // it has itself waited for what came before it (by expert, the route map):
    // the first stages' W is read while x is being quantised and stored.
    if ((int)blockIdx.x < g.units) ahead = min(g.ring, g.stages);
    const uint8_t* wsf = a.wscale + ((size_t)next.expert * (GATED ? 2 : 1) * g.tiles.d + next.tile) * g.stages * 1024;
    for (int s = 0; s < ahead; ++s)
      load_w(s, base + (uint32_t)s * g.stage_bytes, bar0 + s * 8,
             next.expert * (GATED ? 2 * a.N : a.N) + next.tile * 128, wsf, wsf + (size_t)g.tiles.d * g.stages * 1024);
    grid_wait();
  }
  for (int u = blockIdx.x; u < g.units && ok; u += gridDim.x) {
    const MxUnit m = next;
    next = mx_unit<EXPERTS>(a, u + gridDim.x, g.units, g.tiles);
    const int wrow = m.expert * (GATED ? 2 * a.N : a.N) + m.tile * 128;
    const uint8_t* wsf = a.wscale + ((size_t)m.expert * (GATED ? 2 : 1) * g.tiles.d + m.tile) * g.stages * 1024;
    const uint8_t* usf = wsf + (size_t)g.tiles.d * g.stages * 1024;
    const uint8_t* xsf = a.xscale + (size_t)(m.slot0 / a.bn) * g.stages * g.sfb_bytes;
    for (int s = 0; s < g.stages; ++s, ++it, r.next(g.ring)) {
      if (it >= g.ring && !mx_wait_warp(&B.empty[r.slot], r.phase ^ 1, abort, limit)) {
        ok = false;
        break;
      }
      const uint32_t st = base + (uint32_t)r.slot * g.stage_bytes, bar = bar0 + (uint32_t)r.slot * 8;
      if (it >= ahead) load_w(s, st, bar, wrow, wsf, usf);
      if (lead) {
        mx_tma_2d(st + g.a_bytes, &a.xmap, s * 128, m.slot0, bar);
        mx_bulk(st + g.a_bytes + g.b_bytes + g.sfa_bytes, xsf + (uint32_t)s * g.sfb_bytes, g.sfb_bytes, bar);
      }
    }
  }
  return it;
}

// What a CTA that gave up still has in flight ends before its shared and tensor
// memory go: the copies of the last stages loaded, and the MMAs of the last one
// issued. Called when all its warps are done, since any of them may give up
// after the loader and the issuer have left.
__device__ __forceinline__ void mx_drain_copies(MxBars& B, int ring, int loaded) {
  int never = 0;
  for (int i = max(0, loaded - ring); i < loaded; ++i) mbar_wait_abort(&B.full[i % ring], (i / ring) & 1, &never, kMxDrainNs);
}
__device__ __forceinline__ void mx_drain_mmas(MxBars& B, int ring, int issued) {
  int never = 0;
  if (issued > 0) mbar_wait_abort(&B.empty[(issued - 1) % ring], ((issued - 1) / ring) & 1, &never, kMxDrainNs);
}

// (returns the stages whose MMAs it issued)
template <bool GATED, bool EXPERTS, int NRB>
__device__ int mx_issuer(const MxTcArgs& a, const MxGeom& g, MxBars& B, unsigned char* smem, uint32_t tmem,
                         volatile int* abort, uint64_t limit) {
  MxRing r;
  int it = 0, nu = 0;
  bool ok = true;
  constexpr int H = GATED ? 2 : 1;
  const bool lead = mx_elect();
  const uint32_t base = smem_u32(smem);
  if (a.stall_issuer && !mx_wait_warp(&B.never, 0, abort, limit)) return 0;
  MxUnit next = mx_unit<EXPERTS>(a, blockIdx.x, g.units, g.tiles);
  for (int u = blockIdx.x; u < g.units && ok; u += gridDim.x, ++nu) {
    const MxUnit m = next;
    next = mx_unit<EXPERTS>(a, u + gridDim.x, g.units, g.tiles);
    const uint32_t idesc = mx_idesc((m.rows + 15) / 16 * 16);
    const int buf = nu & 1;
    if (nu >= 2 && !mx_wait_warp(&B.acc_empty[buf], ((nu >> 1) - 1) & 1, abort, limit)) break;
    tc_fence_after();
    const uint32_t d = tmem + (uint32_t)(buf * H * a.bn);
    for (int s = 0; s < g.stages; ++s, ++it, r.next(g.ring)) {
      if (!mx_wait_warp(&B.full[r.slot], r.phase, abort, limit)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t st = base + (uint32_t)r.slot * g.stage_bytes;
      const int steps = g.ksteps - s * 4;
      if (steps >= 4)
        mx_issue_stage<GATED, NRB>(st, g.b_bytes, tmem + kMxSfCol, d, (uint32_t)a.bn, idesc, 4, s == 0, lead);
      else
        mx_issue_stage<GATED, NRB>(st, g.b_bytes, tmem + kMxSfCol, d, (uint32_t)a.bn, idesc, steps, s == 0, lead);
      if (lead) tc_commit(&B.empty[r.slot]);
    }
    if (ok && lead) tc_commit(&B.acc_full[buf]);
  }
  return it;
}

template <bool GATED, bool EXPERTS, typename T>
__device__ void mx_epilogue(const MxTcArgs& a, const MxGeom& g, MxBars& B, uint32_t tmem, unsigned char* stage,
                            volatile int* abort, uint64_t limit) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quarter = warp & 3, part = warp >> 2;
  const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
  T* out = static_cast<T*>(a.out);
  const bool words = sizeof(T) == 2 && a.N % 8 == 0 && ((uintptr_t)out) % 16 == 0;
  // the next unit and its rows' places are read while this one is stored: a
  // chain of global loads between two units cost about as much as storing one
  constexpr int kStep = kMxEpiWarps / 4 * 32;  // columns between a warp's pieces of 32
  constexpr int kPieces = (240 + kStep - 1) / kStep;
  int nu = 0, row[kPieces];
  MxUnit next = mx_unit<EXPERTS>(a, blockIdx.x, g.units, g.tiles);
  auto rows_of = [&](const MxUnit& m) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int c = part * 32 + k * kStep + lane;
      row[k] = EXPERTS ? (c < m.rows ? a.route_of_slot[m.slot0 + c] : 0) : m.slot0 + c;
    }
  };
  rows_of(next);
  for (int u = blockIdx.x; u < g.units; u += gridDim.x, ++nu) {
    const MxUnit m = next;
    next = mx_unit<EXPERTS>(a, u + gridDim.x, g.units, g.tiles);
    const int buf = nu & 1;
    const int n = m.tile * 128 + quarter * 32 + lane;
    const bool test = a.stall_epilogue && warp == 0;
    const bool full = mx_wait_warp(test ? &B.never : &B.acc_full[buf], test ? 0 : (nu >> 1) & 1, abort, limit);
    // The four warps of a part meet at its barrier while they store: they go on
    // together or not at all. (One may give up on the abort flag just before the
    // accumulator that its neighbours then find complete.)
    if (!mx_vote_part(full, 1 + part)) return;
    tc_fence_after();
    const uint32_t d = tmem + lane_base + (uint32_t)(buf * (GATED ? 2 : 1) * a.bn);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int c0 = part * 32 + k * kStep;
      if (c0 >= m.rows) break;
      uint32_t v[32], w[32];
      tmem_ld32(d + c0, v);
      if (GATED) tmem_ld32(d + a.bn + c0, w);
      tmem_ld_wait();
      reg_fence32(v);
      if (GATED) reg_fence32(w);
      float y[32];
#pragma unroll
      for (int c = 0; c < 32; ++c)
        y[c] = GATED ? mx_silu(__uint_as_float(v[c])) * __uint_as_float(w[c]) : __uint_as_float(v[c]);
      if (words)
        mx_store32_words<T>(y, out, row[k], m.rows - c0, m.tile * 128, a.N, a.N, stage + part * kMxStoreBytes, 1 + part);
      else
        mx_store32<T>(y, out, row[k], m.rows - c0, n, a.N);
    }
    rows_of(next);
    tc_fence_before();
    if (lane == 0) mbar_arrive(&B.acc_empty[buf]);
    __syncwarp();
  }
}

template <bool GATED, bool EXPERTS, typename T>
__global__ void __launch_bounds__(kMxThreads, 1) k_mx_tc(const __grid_constant__ MxTcArgs a, int ring, FastDiv tiles) {
  extern __shared__ unsigned char mx_smem_raw[];
  __shared__ __align__(8) MxBars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort;
  unsigned char* smem = mx_smem_raw + ((1024u - (smem_u32(mx_smem_raw) & 1023u)) & 1023u);
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);  // (the same for the warp, and known to be)
  if (threadIdx.x == 0) {
    for (int i = 0; i < ring; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], kMxEpiWarps);
    }
    mbar_init(&bars.never, 1);
    s_abort = 0;
    mbar_fence_init();
  }
  if (threadIdx.x == kMxEpiWarps * 32) {
    mx_prefetch_map(&a.wmap);
    mx_prefetch_map(&a.xmap);
  }
  if (warp == 0) tmem_alloc(&tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (the loader alone waits for the kernel before this one: what the others read
  // and write hangs on its copies of x, and the map was complete before)
  grid_launch();
  const uint32_t tmem = tmem_slot;
  volatile int* abort = &s_abort;
  const uint64_t limit = a.wait_ns ? a.wait_ns : kMxWaitNs;
  const MxGeom g = mx_geom<GATED, EXPERTS>(a, ring, tiles);
  int loaded = 0, issued = 0;  // stages, in the warp that did it
  if (g.units == 0) {
    grid_wait();  // (every route was dropped; this kernel still ends after the one before it)
  } else if (warp < kMxEpiWarps) {
    mx_epilogue<GATED, EXPERTS, T>(a, g, bars, tmem, smem + (size_t)ring * g.stage_bytes, abort, limit);
  } else if (warp == kMxEpiWarps) {
    loaded = mx_loader<GATED, EXPERTS>(a, g, bars, smem, abort, limit);
  } else if (warp == kMxEpiWarps + 1) {
    if (a.nrb == 1)
      issued = mx_issuer<GATED, EXPERTS, 1>(a, g, bars, smem, tmem, abort, limit);
    else
      issued = mx_issuer<GATED, EXPERTS, 2>(a, g, bars, smem, tmem, abort, limit);
  }
  tc_fence_before();
  __syncthreads();
  if (*abort) {  // (nobody sets it any more: the same for all)
    mx_drain_copies(bars, ring, loaded);
    mx_drain_mmas(bars, ring, issued);
    if (threadIdx.x == 0) atomicOr(a.err, 2u);
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Rows of codes as bytes, boxes of 128 bytes (256 values) x `box` rows. Box
// starts are multiples of 128 bytes, rows of 16; what lies past a row or the
// last row reads as 0.
cudaError_t mx_code_map(CUtensorMap* m, const uint8_t* codes, long rows, int K, int box) {
  const cuuint64_t bytes = (cuuint64_t)mx_blocks(K) * 16;
  const cuuint64_t dims[2] = {bytes, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {bytes};
  const cuuint32_t boxes[2] = {128, (cuuint32_t)box};
  return tensor_map_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, boxes);
}

template <bool GATED, bool EXPERTS, typename T>
cudaError_t mx_launch(const MxTcArgs& a, cudaStream_t st) {
  auto kern = k_mx_tc<GATED, EXPERTS, T>;
  static OncePerDevice done;
  const cudaError_t limit = allow_smem(done, kern, (int)kMxSmem);
  if (limit != cudaSuccess) return limit;
  const uint32_t stage = (uint32_t)(GATED ? 2 : 1) * (kMxTileBytes + 1024) + (uint32_t)a.bn * 128 + (uint32_t)a.nrb * 1024;
  const uint32_t stage_bytes = (stage + 1023) / 1024 * 1024;
  const uint32_t store = kMxEpiWarps / 4 * kMxStoreBytes;
  const int ring = (int)std::min<uint32_t>(kMxMaxStages, (kMxSmem - 1024 - store) / stage_bytes);
  const long units = (long)a.max_blocks * ((a.N + 127) / 128);
  const int grid = (int)std::max<long>(1, std::min<long>(units, a.sms));
  return launch_after(kern, dim3(grid), kMxThreads, 1024 + ring * stage_bytes + store, st, a, ring,
                         FastDiv((a.N + 127) / 128));
}

// One thread a 4-byte word of the laid-out scales; absent rows and blocks get 0.
__global__ void __launch_bounds__(256) k_mx_weight_scales(const uint8_t* __restrict__ s, int halves, int N, int nb,
                                                          int tiles, int chunks, long words, uint32_t* __restrict__ out) {
  for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += (long)gridDim.x * blockDim.x) {
    const int w = (int)(i & 127);
    long j = i >> 7;
    const int c = (int)(j % chunks);
    j /= chunks;
    const int tile = (int)(j % tiles);
    const long eh = j / tiles;  // expert * halves + half
    const int n = tile * 128 + (w & 3) * 32 + (w >> 2);
    uint32_t v = 0;
    if (n < N)
      for (int b = 0; b < 4; ++b)
        if (c * 4 + b < nb) v |= (uint32_t)s[((size_t)eh * N + n) * nb + c * 4 + b] << (8 * b);
    out[i] = v;
  }
}

// A warp takes up to kRqUnroll times 256 columns (eight blocks, four lanes
// each) of a row of x, all loads in flight at once. Dense (no slots): the first
// thread clears the error word. By expert: the route map is the kernel before
// this one in the stream, and it lets this one start only after it has itself
// waited for all that came before it, so x may be read, and quantised, while
// the map is being made; only the slots wait for it. 2048 x 4096 bf16: 4 us;
// 32768 x 1536: 24 us = 5.3 TB/s, bound by its instructions and the memory alike.
constexpr int kRqUnroll = 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(256, VEC && sizeof(T) == 2 ? 8 : 5)
    k_mx_rows_quantize(const MxQuantArgs a, int stages, int per, FastDiv segs, FastDiv bn, int items) {
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);
  if (!a.slot_of_route || i >= items) grid_wait();
  if (!a.slot_of_route && blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0u;
  if (!a.slot_of_route || i >= items) grid_launch();
  if (i >= items) return;
  const int nb = mx_blocks(a.K);
  const int row = (int)segs.div(i), s0 = (i - row * (int)segs.d) * per, n = min(per, stages - s0);
  const T* x = static_cast<const T*>(a.x) + (size_t)row * a.ld + s0 * 256 + lane * 8;
  const int left = a.K - s0 * 256 - lane * 8;
  Eight<T, VEC> e[kRqUnroll];
#pragma unroll
  for (int u = 0; u < kRqUnroll; ++u) e[u].load(x + u * 256, u < n ? max(0, min(8, left - u * 256)) : 0);
  uint32_t q[kRqUnroll], byte[kRqUnroll];
#pragma unroll
  for (int u = 0; u < kRqUnroll; ++u) {
    q[u] = byte[u] = 0;
    if (u < n) {
      float v[8];
      e[u].to(v);
      q[u] = mxfp4_codes(v, e[u].block_amax_bits(), byte[u]);
    }
  }
  // Few and wide stores, since a row goes to all its routes' slots (against eight
  // stores of four bytes or one for each slot: 18.4 us instead of 19.2 a call at
  // 10 routes a row, 25.8 instead of 26.7 at 8, and 189.5 instead of 188.4 at one
  // route a row, where nothing pays for the exchange): the codes of four neighbouring
  // lanes change places, so that lane l has the 16 bytes of block l of these
  // columns; lane u + 16 c has the four scale bytes of stage u, chunk c.
  static_assert(kRqUnroll == 4, "a lane of four for a stage");
  {
    const bool odd = lane & 1, high = lane & 2;
    uint32_t x0 = __shfl_xor_sync(0xFFFFFFFFu, odd ? q[0] : q[1], 1);
    uint32_t x1 = __shfl_xor_sync(0xFFFFFFFFu, odd ? q[2] : q[3], 1);
    (odd ? q[0] : q[1]) = x0;
    (odd ? q[2] : q[3]) = x1;
    x0 = __shfl_xor_sync(0xFFFFFFFFu, high ? q[0] : q[2], 2);
    x1 = __shfl_xor_sync(0xFFFFFFFFu, high ? q[1] : q[3], 2);
    (high ? q[0] : q[2]) = x0;
    (high ? q[1] : q[3]) = x1;
    const int from = (lane & 7) * 4 + (lane >> 3);
#pragma unroll
    for (int u = 0; u < kRqUnroll; ++u) q[u] = __shfl_sync(0xFFFFFFFFu, q[u], from);
  }
  uint32_t word = byte[0];
  word = (lane & 3) == 1 ? byte[1] : word;
  word = (lane & 3) == 2 ? byte[2] : word;
  word = (lane & 3) == 3 ? byte[3] : word;
  word <<= lane * 2 & 24;
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 8);
  int mine = row;  // lane j: the slot of the row's route j (at most 32)
  if (a.slot_of_route) {
    grid_wait();
    grid_launch();  // (only now: the products' kernel relies on the map when it starts)
    mine = lane < a.topk ? a.slot_of_route[row * a.topk + lane] : -1;
  }
  const bool code_on = lane < n * 8 && s0 * 8 + lane < nb;
  const bool scale_on = (lane & 12) == 0 && (lane & 3) < n;
  for (int j = 0; j < a.topk; ++j) {
    const int r = row * a.topk + j;
    const int slot = __shfl_sync(0xFFFFFFFFu, mine, j);
    if (slot < 0) {
      if (s0 == 0) {
        char* o = static_cast<char*>(a.out) + (size_t)r * a.out_row_bytes;
        for (int b = lane * 2; b < a.out_row_bytes; b += 64) *reinterpret_cast<uint16_t*>(o + b) = 0;
      }
      continue;
    }
    const int b = (int)bn.div(slot), t = slot - b * (int)bn.d;
    if (code_on)
      *reinterpret_cast<uint4*>(a.codes + ((size_t)slot * nb + s0 * 8 + lane) * 16) =
          make_uint4(q[0], q[1], q[2], q[3]);
    if (scale_on)
      *reinterpret_cast<uint32_t*>(
          a.scales + ((((size_t)b * stages + s0 + (lane & 3)) * 2 + (lane >> 4)) * a.nrb + (t >> 7)) * 512 +
          (t & 31) * 16 + ((t & 127) >> 5) * 4) = word;
  }
}

// Route map for the block kernel, by one cluster of kMapCtas CTAs: every CTA
// counts its part of the routes by expert in shared memory, reads the others'
// counts, and places its routes. Their order within an expert is that of the
// atomics, which no result depends on: a row's product is the same in any
// place of any block. Writes the blocks' experts and rows and the number of
// blocks, slot_of_route (-1: no such expert), route_of_slot (only for slots
// with a route) and the error word. 16384 routes: 5 us; the three launches of the
// stable map that the trellis layer uses take 9 us.
constexpr int kMapCtas = 8;
constexpr int kMapThreads = 1024;

// Up to kMapHeld routes of a thread stay in registers between the two passes;
// more go through slot_of_route.
constexpr int kMapHeld = 4;

__device__ __forceinline__ int map_peer_int(const int* p, int rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];\n" : "=r"(v) : "r"(at) : "memory");
  return v;
}

__global__ void __cluster_dims__(kMapCtas, 1, 1) __launch_bounds__(kMapThreads) k_mx_map(const MxMapArgs a) {
  __shared__ int s_cnt[kMaxExperts];    // this CTA's routes by expert
  __shared__ int s_base[kMaxExperts];   // slot of this CTA's first route of the expert
  __shared__ int s_warp[kMaxExperts / 32];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  for (int e = tid; e < kMaxExperts; e += kMapThreads) s_cnt[e] = 0;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  grid_wait();
  grid_launch();
  const int part = (a.R + kMapCtas - 1) / kMapCtas, lo = (int)rank * part, hi = min(a.R, lo + part);
  const bool held = part <= kMapHeld * kMapThreads;
  int e[kMapHeld], at[kMapHeld];
  for (int r0 = lo + tid; r0 < hi; r0 += kMapThreads * kMapHeld) {
#pragma unroll
    for (int u = 0; u < kMapHeld; ++u) e[u] = r0 + u * kMapThreads < hi ? a.ids[r0 + u * kMapThreads] : 0;
#pragma unroll
    for (int u = 0; u < kMapHeld; ++u) {
      const int r = r0 + u * kMapThreads;
      at[u] = -1;
      if (r < hi) {
        if (e[u] >= 0 && e[u] < a.E)
          at[u] = atomicAdd(&s_cnt[e[u]], 1);
        else
          s_bad = 1;
        if (!held) a.slot_of_route[r] = at[u];  // the place among this CTA's, for now
      }
    }
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  // thread x: this CTA's base within expert x, and the expert's total
  int before = 0, total = 0, blocks = 0;
  if (tid < a.E) {
#pragma unroll
    for (int c = 0; c < kMapCtas; ++c) {
      const int v = map_peer_int(&s_cnt[tid], c);
      if (c < (int)rank) before += v;
      total += v;
    }
    blocks = (total + a.bn - 1) / a.bn;
  }
  const int bad = __syncthreads_or(rank == 0 && tid < kMapCtas ? map_peer_int(&s_bad, tid) : 0);
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");  // (done with the peers' counts)
  int incl = blocks;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31 && warp < kMaxExperts / 32) s_warp[warp] = incl;
  __syncthreads();
  if (tid < a.E) {
    int first = incl - blocks;
    for (int w = 0; w < warp; ++w) first += s_warp[w];
    s_base[tid] = first * a.bn + before;
    if (rank == 0) {
      for (int b = 0; b < blocks; ++b) a.block_info[first + b] = make_int2(tid, min(a.bn, total - b * a.bn));
      if (tid == a.E - 1) *a.nblocks = first + blocks;
    }
  }
  if (rank == 0 && tid == 0) *a.err = bad ? 1u : 0u;
  __syncthreads();
  for (int r0 = lo + tid; r0 < hi; r0 += kMapThreads * kMapHeld) {
    if (!held) {
#pragma unroll
      for (int u = 0; u < kMapHeld; ++u) {
        const int r = r0 + u * kMapThreads;
        e[u] = r < hi ? a.ids[r] : 0;
        at[u] = r < hi ? a.slot_of_route[r] : -1;
      }
    }
#pragma unroll
    for (int u = 0; u < kMapHeld; ++u) {
      const int r = r0 + u * kMapThreads;
      if (r >= hi) break;
      const int slot = at[u] < 0 ? -1 : s_base[e[u]] + at[u];
      a.slot_of_route[r] = slot;
      if (slot >= 0) a.route_of_slot[slot] = r;
    }
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");  // no CTA leaves while another reads its counts
}

}  // namespace

size_t mx_weight_scale_bytes(int E, int halves, int N, int K) {
  return (size_t)E * halves * ((N + 127) / 128) * mx_stages(K) * 1024;
}

cudaError_t launch_mx_weight_scales(const uint8_t* scales, int E, int halves, int N, int K, uint8_t* out,
                                    cudaStream_t st) {
  const long words = (long)(mx_weight_scale_bytes(E, halves, N, K) / 4);
  const int ctas = (int)std::min<long>(152 * 16, (words + 255) / 256);
  k_mx_weight_scales<<<ctas, 256, 0, st>>>(scales, halves, N, mx_blocks(K), (N + 127) / 128, 2 * mx_stages(K), words,
                                           reinterpret_cast<uint32_t*>(out));
  return cudaGetLastError();
}

cudaError_t mx_weight_map(CUtensorMap* m, const uint8_t* codes, long rows, int K) {
  return mx_code_map(m, codes, rows, K, 128);
}

cudaError_t launch_mx_tc(MxTcArgs& a, const uint8_t* codes_x, long slots, int out_dtype, cudaStream_t st) {
  const cudaError_t e = mx_code_map(&a.xmap, codes_x, slots, a.K, a.bn);
  if (e != cudaSuccess) return e;
  auto go = [&](auto elem) {
    using T = decltype(elem);
    if (a.block_info) return a.gated ? mx_launch<true, true, T>(a, st) : mx_launch<false, true, T>(a, st);
    return a.gated ? mx_launch<true, false, T>(a, st) : mx_launch<false, false, T>(a, st);
  };
  return TM_BY_DTYPE(out_dtype, go);
}

cudaError_t launch_mx_map(const MxMapArgs& a, cudaStream_t st) {
  return launch_after(k_mx_map, dim3(kMapCtas), kMapThreads, 0, st, a);
}

cudaError_t launch_mx_rows_quantize(const MxQuantArgs& a, int dtype, cudaStream_t st) {
  const int es = dtype_bytes(dtype);
  const int stages = mx_stages(a.K), segs = (stages + kRqUnroll - 1) / kRqUnroll, per = (stages + segs - 1) / segs;
  const int items = a.x_rows * segs;
  auto go = [&](auto elem, auto vec) {
    return launch_after(k_mx_rows_quantize<decltype(elem), decltype(vec)::value>, dim3((items + 7) / 8), 256, 0, st, a,
                           stages, per, FastDiv(segs), FastDiv(a.bn), items);
  };
  return TM_BY_DTYPE_VEC(dtype, eights(a.x, a.ld, a.K, es), go);
}

}  // namespace tmoe
