// Storing accumulator tiles whose lanes are output channels and whose columns
// are rows of the result (tensor-core epilogues).
#pragma once

#include <stdint.h>

#include "elem.cuh"

namespace tmoe {

// 32 columns (rows of y) of a thread's channel, as T: y[c] for row `row` of
// lane c, `rows` of them.
template <typename T>
__device__ __forceinline__ void mx_store32(const float (&y)[32], T* __restrict__ out, int row, int rows, int n, int N) {
  T* o = out + n;
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    const int r = __shfl_sync(0xFFFFFFFFu, row, c);
    if (n < N && c < rows) o[(size_t)r * N] = from_f32<T>(y[c]);
  }
}

// The same for 16-bit types where rows of y are whole 16-byte words, channels
// `first` to `end` (at most 128): the four warps of a piece put 16 rows at a time into shared memory and
// store them from there in 16-byte words, a whole row's 256 bytes by 16 lanes
// (as single elements a warp's store covered 64 bytes, and storing a piece of
// 32 rows took 1400 cycles). Neighbouring lanes first swap halves, so that the
// even one holds both channels of an even row and the odd one of the next; the
// 64-byte halves of odd rows change places, which keeps the two apart in banks.
template <typename T>
__device__ __forceinline__ void mx_store32_words(const float (&y)[32], T* __restrict__ out, int row, int rows, int first,
                                                 int end, int N, unsigned char* stage, int bar) {
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, odd = lane & 1;
  const uint32_t pick = odd ? 0x3276u : 0x5410u;
  const int t = quarter * 32 + lane, chunk = t & 15;
  const bool in = first + chunk * 8 < end;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h * 16 >= rows) break;
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
      uint32_t p;
      T* e = reinterpret_cast<T*>(&p);
      e[0] = from_f32<T>(y[h * 16 + c]);
      e[1] = from_f32<T>(y[h * 16 + c + 1]);
      const uint32_t q = __shfl_xor_sync(0xFFFFFFFFu, p, 1);
      const int word = (quarter * 16 + (lane >> 1)) ^ (odd << 4);
      *reinterpret_cast<uint32_t*>(stage + (c + odd) * 256 + word * 4) = __byte_perm(p, q, pick);
    }
    asm volatile("bar.sync %0, 128;\n" ::"r"(bar) : "memory");
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = k * 8 + (t >> 4);
      const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 256 + ((chunk * 16) ^ ((r & 1) << 6)));
      const int to = __shfl_sync(0xFFFFFFFFu, row, h * 16 + r);
      if (in && h * 16 + r < rows)
        *reinterpret_cast<uint4*>(out + (size_t)to * N + first + chunk * 8) = v;
    }
    asm volatile("bar.sync %0, 128;\n" ::"r"(bar) : "memory");
  }
}

// Whether all four warps of a part say yes, by its named barrier.
__device__ __forceinline__ bool mx_vote_part(bool yes, int bar) {
  uint32_t all;
  asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.and.pred q, %2, 128, p;\nselp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(all)
               : "r"((uint32_t)yes), "r"(bar)
               : "memory");
  return all != 0;
}

}  // namespace tmoe
