// Shared by the tensor-core kernels with MXFP4 operands: copies, scales and the
// `tcgen05.mma.kind::mxf4` of one pipeline stage (256 columns).
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "pdl.cuh"
#include "tc.cuh"

namespace tmoe {

constexpr uint64_t kMxWaitNs = 2000000000ull;   // limit of a pipeline wait
constexpr uint64_t kMxDrainNs = 500000000ull;   // of a wait for copies in flight after one gave up
constexpr int kMxTileBytes = 128 * 128;         // 128 rows of W, 256 columns

// silu(g) = g / (1 + exp(-g)) with the hardware's exp2 and reciprocal (each a
// few ulp). Subnormals flush: an exp(-g) that small leaves 1, and a reciprocal
// that small (g below -87) makes the result 0. Written out because the same
// through __expf and __fdividef also scales subnormals, and the epilogue of a
// gated block of 112 rows is bound by its instructions.
__device__ __forceinline__ float mx_silu(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return g * r;
}

__device__ __forceinline__ void mx_prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(m) : "memory");
}

// The copies of a stage take shared addresses, which a converged warp keeps in
// uniform registers (from one thread's own branch, issuing a stage's copies took
// 280-400 cycles).
__device__ __forceinline__ void mx_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mx_tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n"
               ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void mx_bulk(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// 512 bytes of scales (32 rows of 16 bytes, rows 16 bytes apart) to four
// columns of tensor memory, repeated in each quarter of the lanes.
__device__ __forceinline__ void mx_copy_scales(uint32_t taddr, uint32_t saddr) {
  const uint64_t desc = smem_desc(saddr, 128, 128);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
}

// D (+)= A B^T over 64 columns with one scale per 32.
__device__ __forceinline__ void mx_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc));
}

// Instruction descriptor: E2M1 x E2M1, E8M0 scales, fp32 accumulator, both
// operands K-major, M = 128. Bits 4 and 29 take the first of the two scale
// bytes used (0 or 2 of the chunk's four).
__device__ __forceinline__ uint32_t mx_idesc(int n) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(128 >> 4) << 24);
}

// One thread of a converged warp.
__device__ __forceinline__ bool mx_elect() {
  uint32_t p;
  asm volatile("{\n.reg .pred q;\nelect.sync _|q, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}

// mbar_wait_abort by a whole warp, with one answer for it.
__device__ __forceinline__ bool mx_wait_warp(uint64_t* mbar, uint32_t parity, volatile int* abort, uint64_t limit) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_abort(mbar, parity, abort, limit));
}

// Position in the ring of stages: slot and the parity of its use.
struct MxRing {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int ring) {
    if (++slot == ring) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// The MMAs of one stage: the chunks' scales to tensor memory, then one MMA per
// 64 columns (`steps` of them) and half. The stage holds the W tile(s), the x
// tile (b_bytes), the W scales and the x scales; `tsfa` is the first of the
// 8 H + 8 NRB columns of tensor memory for scales. Run by a whole warp, of which `lead`
// is one thread: the operands are then the same for the warp, which keeps them
// in uniform registers; issued from a single thread's branch, each
// instruction cost 110-120 cycles of moving its operands there.
template <bool GATED, int NRB>
__device__ __forceinline__ void mx_issue_stage(uint32_t st, uint32_t b_bytes, uint32_t tsfa, uint32_t d, uint32_t dup,
                                               uint32_t idesc, int steps, bool first, bool lead) {
  constexpr int H = GATED ? 2 : 1;
  const uint32_t sfa = st + H * kMxTileBytes + b_bytes, sfb = sfa + H * 1024;
  const uint32_t tsfb = tsfa + 8u * H;
  const uint64_t adesc = smem_desc_sw128(st), bdesc = smem_desc_sw128(st + H * kMxTileBytes);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if (c * 2 < steps) {
#pragma unroll
      for (int h = 0; h < H; ++h)
        if (lead) mx_copy_scales(tsfa + (uint32_t)(c * H + h) * 4, sfa + h * 1024 + c * 512);
#pragma unroll
      for (int r = 0; r < NRB; ++r)
        if (lead) mx_copy_scales(tsfb + (uint32_t)(c * NRB + r) * 4, sfb + (uint32_t)(c * NRB + r) * 512);
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k < steps) {
#pragma unroll
      for (int h = 0; h < H; ++h)
        if (lead)
          mx_mma(d + (h ? dup : 0u), adesc + (uint64_t)(h * (kMxTileBytes >> 4) + k * 2), bdesc + (uint64_t)(k * 2),
                 idesc | ((uint32_t)((k & 1) * 2) << 4) | ((uint32_t)((k & 1) * 2) << 29),
                 tsfa + (uint32_t)((k >> 1) * H + h) * 4, tsfb + (uint32_t)((k >> 1) * NRB) * 4,
                 !first || k > 0 ? 1u : 0u);
    }
  }
}

}  // namespace tmoe
