// Products with MXFP4 weights for few rows (sm_103a): one launch that reads the
// touched weights once, split along K over the CTAs of a cluster.
//
// A unit is 128 output channels (gated: the 128 gate and the 128 up rows) and a
// chunk of up to 16 rows of one expert; each CTA of the unit's cluster takes
// a contiguous part of the 256-column stages. The W tile and its scales come by
// TMA; the rows of x are quantised by four warps straight into the swizzled
// operand and scale layout in shared memory, so there is no pass over x before.
// Nor is there a row map: the chunk with index r starts at route r, and exists
// if the number of earlier routes of the same expert is a multiple of 16; its
// rows are that route and the next ones of the expert. Each warp finds that by
// itself with a ballot for every 32 ids, and the CTAs without a chunk leave.
// The MMA is the block-scaled one of mxfp4_mma.cuh with the rows of x as
// N = 16 columns; tensor cores have time to spare here, what bounds the call is
// the weights' bytes and the latency of one load, MMA and drain chain, which
// the split shortens and spreads over the SMs.
//
// The partial sums of a unit are sent to the CTA of the cluster that owns their
// row, which adds them in rank order: the same bits every time. A CTA frees its
// tensor memory before it waits for its cluster, so that a CTA that waits holds
// nothing that another one needs.
//
// One token, 4096 x 4096: 6.8 us a call back to back, of which the kernel's chain
// is 3.4 us (setup 0.35, first W tile and x in shared memory 1.0, second stage
// and MMA 0.5, drain 0.1, cluster 0.9, sums and store 0.5) and the weights'
// bytes 1.3 us. 8 tokens x 8 of 128 experts, gated 1024 -> 512: 6.8 us, bytes
// 4.2 us. Held back by latency and launch, not by bytes or instructions.
#include <algorithm>

#include "elem.cuh"
#include "mxfp4.cuh"
#include "mxfp4.h"
#include "mxfp4_mma.cuh"
#include "status.h"

namespace tmoe {

namespace {

constexpr int kMdThreads = 192;  // four warps quantise and drain, one loads, one issues
constexpr int kMdMaxRing = 8;
constexpr int kMdXBytes = kMxDecRows * 128;  // the x tile of a stage

struct MdBars {
  uint64_t full[kMdMaxRing], empty[kMdMaxRing];
  uint64_t acc;
  uint64_t never;  // nothing arrives on it (test of the bounded waits)
};

__device__ __forceinline__ uint32_t md_cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void md_cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void md_cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }
__device__ __forceinline__ uint32_t md_peer(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ void md_peer_store(uint32_t a, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(a), "f"(v) : "memory");
}

// Quantises eight values of a row of x in any of the element types (n of them
// exist; the four lanes of a block together).
__device__ __forceinline__ uint32_t md_quantize(const MxDecArgs& a, size_t off, int n, uint32_t& byte) {
  auto get = [&](auto elem, auto vec) {
    using T = decltype(elem);
    Eight<T, decltype(vec)::value> e;
    e.load(static_cast<const T*>(a.x) + off, n);
    float v[8];
    e.to(v);
    return mxfp4_codes(v, e.block_amax_bits(), byte);
  };
  return TM_BY_DTYPE_VEC(a.x_dtype, a.vec, get);
}

__device__ __forceinline__ void md_store(const MxDecArgs& a, size_t i, float y) {
  if (a.out_dtype == TM_F32)
    static_cast<float*>(a.out)[i] = y;
  else if (a.out_dtype == TM_BF16)
    static_cast<__nv_bfloat16*>(a.out)[i] = from_f32<__nv_bfloat16>(y);
  else
    static_cast<__half*>(a.out)[i] = from_f32<__half>(y);
}

// The rows of the chunk that starts at route r0: `expert` (out of range: none),
// `rows` of them (0: no chunk starts here). Called by each warp; `list` (one
// warp's) gets the routes.
struct MdChunk {
  int expert, rows;
  bool bad;  // some id is out of range
};

__device__ __forceinline__ MdChunk md_find(const MxDecArgs& a, int r0, int* list) {
  const int lane = threadIdx.x & 31;
  MdChunk m;
  m.expert = a.ids[r0];
  m.bad = false;
  int before = 0, from = 0;
  for (int i = 0; i < a.rows; i += 128) {
    int id[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) id[u] = i + u * 32 + lane < a.rows ? a.ids[i + u * 32 + lane] : 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = i + u * 32 + lane;
      m.bad |= id[u] < 0 || id[u] >= a.E;
      const bool is = r < a.rows && id[u] == m.expert;
      const uint32_t lo = __ballot_sync(0xFFFFFFFFu, is && r < r0), hi = __ballot_sync(0xFFFFFFFFu, is && r >= r0);
      const int at = from + __popc(hi & ((1u << lane) - 1u));
      if (list && is && r >= r0 && at < kMxDecRows) list[at] = r;
      before += __popc(lo);
      from += __popc(hi);
    }
  }
  m.rows = before % kMxDecRows == 0 ? min(kMxDecRows, from) : 0;
  return m;
}

template <bool GATED>
__global__ void __launch_bounds__(kMdThreads) k_mx_dec(const __grid_constant__ MxDecArgs a, int lsplit, int per, int ring,
                                                       uint32_t cols) {
  constexpr int H = GATED ? 2 : 1;
  const int split = 1 << lsplit;
  extern __shared__ unsigned char md_smem_raw[];
  __shared__ __align__(8) MdBars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort;
  __shared__ int s_row[kMxDecRows];
  unsigned char* smem = md_smem_raw + ((1024u - (smem_u32(md_smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int rank = split > 1 ? (int)md_cluster_rank() : 0;
  const int unit = blockIdx.x >> lsplit;
  const int tiles = (a.N + 127) / 128;
  const int chunk = unit / tiles, tile = unit - chunk * tiles;
  const int stages = mx_stages(a.K);
  const int s_lo = rank * per, s_hi = min(stages, s_lo + per);
  constexpr uint32_t kStage = H * (kMxTileBytes + 1024) + kMdXBytes + 1024;
  static_assert(kStage % 1024 == 0, "operands at multiples of the swizzle atom");
  float* part = reinterpret_cast<float*>(smem + (size_t)ring * kStage);  // [split][H][16 / split][128]

  if (split > 1) md_cluster_arrive();  // (waited for before the first store to a peer)
  if (tid == 128) {
    mx_prefetch_map(&a.wmap);
    for (int i = 0; i < ring; ++i) {
      mbar_init(&bars.full[i], 5);  // the loader's expect_tx and four quantising warps
      mbar_init(&bars.empty[i], 1);
    }
    mbar_init(&bars.acc, 1);
    mbar_init(&bars.never, 1);
    s_abort = 0;
    mbar_fence_init();
  }
  grid_wait();
  grid_launch();
  MdChunk m{0, min(kMxDecRows, a.rows - chunk * kMxDecRows), false};
  if (a.ids) {
    m = md_find(a, chunk, warp == 0 ? s_row : nullptr);
    // (every CTA sees all ids; the first one writes the error word, long
    // before a wait of any CTA can run out and set its bit)
    if (blockIdx.x == 0 && warp == 0) {
      const bool any = __any_sync(0xFFFFFFFFu, m.bad);
      if (lane == 0) *a.err = any ? 1u : 0u;
    }
    if (m.expert < 0 || m.expert >= a.E) {  // a route without an expert gets a row of zeros
      if (rank == 0)
        for (int n = tile * 128 + tid; n < min(a.N, tile * 128 + 128); n += kMdThreads)
          md_store(a, (size_t)chunk * a.N + n, 0.0f);
      return;
    }
  } else if (blockIdx.x == 0 && tid == 0) {
    *a.err = 0u;
  }
  if (m.rows <= 0) return;  // (here and above: the same for the whole cluster)
  if (warp == 5) tmem_alloc(&tmem_slot, cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t tsfa = tmem + (uint32_t)(H * kMxDecRows);
  volatile int* abort = &s_abort;
  const uint64_t limit = a.wait_ns ? a.wait_ns : kMxWaitNs;
  int loaded = 0;  // stages, in the loading warp

  if (warp == 4) {
    const bool lead = mx_elect();
    const uint32_t base = smem_u32(smem), bar0 = smem_u32(&bars.full[0]);
    const int wrow = m.expert * H * a.N + tile * 128;
    const uint8_t* wsf = a.wscale + ((size_t)m.expert * H * tiles + tile) * stages * 1024;
    const uint8_t* usf = wsf + (size_t)tiles * stages * 1024;
    MxRing r;
    int it = 0;
    for (int s = s_lo; s < s_hi; ++s, ++it, r.next(ring)) {
      if (it >= ring && !mx_wait_warp(&bars.empty[r.slot], r.phase ^ 1, abort, limit)) break;
      const uint32_t st = base + (uint32_t)r.slot * kStage, sf = st + H * kMxTileBytes + kMdXBytes;
      const uint32_t bar = bar0 + (uint32_t)r.slot * 8;
      if (lead) {
        mx_expect(bar, H * (kMxTileBytes + 1024));
        mx_tma_2d(st, &a.wmap, s * 128, wrow, bar);
        if (GATED) mx_tma_2d(st + kMxTileBytes, &a.wmap, s * 128, wrow + a.N, bar);
        mx_bulk(sf, wsf + s * 1024, 1024, bar);
        if (GATED) mx_bulk(sf + 1024, usf + s * 1024, 1024, bar);
      }
    }
    loaded = it;
  } else if (warp == 5) {
    const bool lead = mx_elect();
    const uint32_t base = smem_u32(smem), idesc = mx_idesc(kMxDecRows);
    const int ksteps = (mx_blocks(a.K) + 1) / 2;
    MxRing r;
    if (a.stall_issuer) mx_wait_warp(&bars.never, 0, abort, limit);
    for (int s = s_lo; s < s_hi && !*abort; ++s, r.next(ring)) {
      if (!mx_wait_warp(&bars.full[r.slot], r.phase, abort, limit)) break;
      tc_fence_after();
      mx_issue_stage<GATED, 1>(base + (uint32_t)r.slot * kStage, kMdXBytes, tsfa, tmem, (uint32_t)kMxDecRows, idesc,
                               min(4, ksteps - s * 4), s == s_lo, lead);
      if (lead) tc_commit(&bars.empty[r.slot]);
    }
    if (lead) tc_commit(&bars.acc);
  } else {
    MxRing r;
    int it = 0, item = 0;
    for (int s = s_lo; s < s_hi; ++s, ++it, r.next(ring)) {
      if (it >= ring && !mx_wait_warp(&bars.empty[r.slot], r.phase ^ 1, abort, limit)) break;
      unsigned char* st = smem + (size_t)r.slot * kStage;
      unsigned char* bt = st + H * kMxTileBytes;
      unsigned char* sf = bt + kMdXBytes + H * 1024;
      for (int i = 0; i < m.rows; ++i, ++item) {
        if ((item & 3) != warp) continue;
        const int row = a.ids ? s_row[i] : chunk * kMxDecRows + i;
        const int xr = row / a.topk, col = s * 256 + lane * 8;
        uint32_t byte;
        const uint32_t q = md_quantize(a, (size_t)xr * a.ld + col, max(0, min(8, a.K - col)), byte);
        const int g = lane & 16;
        uint32_t word = byte;
        word |= __shfl_sync(0xFFFFFFFFu, byte, g + 4) << 8;
        word |= __shfl_sync(0xFFFFFFFFu, byte, g + 8) << 16;
        word |= __shfl_sync(0xFFFFFFFFu, byte, g + 12) << 24;
        *reinterpret_cast<uint32_t*>(bt + sw128_off(i, lane >> 2) + (lane & 3) * 4) = q;
        if ((lane & 15) == 0)
          *reinterpret_cast<uint32_t*>(sf + (lane >> 4) * 512 + i * 16) = word;
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.full[r.slot]);
    }
  }
  if (split > 1) md_cluster_wait();  // every CTA of the cluster has started
  const int own = kMxDecRows >> lsplit;      // rows that a CTA of the cluster may own: c = rank, rank + split, ...
  if (warp < 4 && s_hi > s_lo) {
    const bool ok = mx_wait_warp(a.stall_epilogue && warp == 0 ? &bars.never : &bars.acc, 0, abort, limit);
    tc_fence_after();
    if (ok) {
      const uint32_t lb = tmem + ((uint32_t)(warp * 32) << 16);
      const uint32_t to = smem_u32(part) + (uint32_t)(rank * H * own * 128 + warp * 32 + lane) * 4;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float v[16];
        tmem_ld16(lb + (uint32_t)(h * kMxDecRows), v);
#pragma unroll
        for (int c = 0; c < kMxDecRows; ++c) {
          if (c >= m.rows) break;
          const uint32_t at = to + (uint32_t)(h * own + (c >> lsplit)) * 512;
          if (split > 1)
            md_peer_store(md_peer(at, (uint32_t)(c & (split - 1))), v[c]);
          else
            part[(size_t)(h * own + c) * 128 + warp * 32 + lane] = v[c];
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort) {  // (nobody sets it any more: the same for all)
    // What is in flight ends before shared and tensor memory go. Here, since any
    // warp may give up after the loader and the issuer are done. (full[] also
    // counts the quantisers' arrivals, one for every stage they reach; a copy
    // in flight lands within the limit.)
    int never = 0;
    for (int i = max(0, loaded - ring); i < loaded; ++i)
      mbar_wait_abort(&bars.full[i % ring], (i / ring) & 1, &never, kMxDrainNs / kMdMaxRing);
    never = 0;
    if (warp == 5) mx_wait_warp(&bars.acc, 0, &never, kMxDrainNs);
    if (tid == 0) atomicOr(a.err, 2u);
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, cols);
  if (split > 1) {
    md_cluster_arrive();
    md_cluster_wait();
  }
  // the sums of the ranks that had stages, in order
  const int active = (stages + per - 1) / per;
  for (int i = tid; i < 128 * ((m.rows - rank + split - 1) >> lsplit); i += kMdThreads) {
    const int n = i & 127, o = i >> 7, c = (o << lsplit) + rank;
    float y[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      y[h] = part[(h * own + o) * 128 + n];
      for (int k = 1; k < active; ++k) y[h] += part[((k * H + h) * own + o) * 128 + n];
    }
    const float v = GATED ? mx_silu(y[0]) * y[H - 1] : y[0];
    const int ch = tile * 128 + n;
    if (ch < a.N) md_store(a, (size_t)(a.ids ? s_row[c] : chunk * kMxDecRows + c) * a.N + ch, v);
  }
}

template <bool GATED>
cudaError_t md_launch(const MxDecArgs& a, int chunks, cudaStream_t st) {
  constexpr int H = GATED ? 2 : 1;
  auto kern = k_mx_dec<GATED>;
  constexpr int kSmem = 104 * 1024;
  static OncePerDevice done;
  const cudaError_t limit = allow_smem(done, kern, kSmem);
  if (limit != cudaSuccess) return limit;
  const int stages = mx_stages(a.K), tiles = (a.N + 127) / 128;
  const int units = chunks * tiles;
  const int lsplit = mx_dec_split(units, stages, a.sms);
  const int split = 1 << lsplit;
  const int per = (stages + split - 1) / split;
  const int stage = H * (kMxTileBytes + 1024) + kMdXBytes + 1024;
  const int part = H * kMxDecRows * 128 * 4;
  // a ring that leaves room for two CTAs on an SM
  const int ring = std::max(1, std::min(std::min(kMdMaxRing, per), (100 * 1024 - part) / stage));
  uint32_t cols = 32;
  while (cols < (uint32_t)(H * kMxDecRows + 8 * H + 8)) cols *= 2;
  const int smem = 1024 + ring * stage + part;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(units * split));
  cfg.blockDim = dim3(kMdThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {(unsigned)split, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a, lsplit, per, ring, cols);
}

}  // namespace

cudaError_t launch_mx_dec(const MxDecArgs& a, int chunks, cudaStream_t st) {
  return a.gated ? md_launch<true>(a, chunks, st) : md_launch<false>(a, chunks, st);
}

}  // namespace tmoe
