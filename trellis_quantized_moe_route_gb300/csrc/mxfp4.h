// Internal launchers of the MXFP4 kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace tmoe {

// Blocks of 32 along K, and the pieces the tensor-core kernels walk: a scale
// chunk covers 128 columns, a pipeline stage 256 (the last one filled up).
__host__ __device__ inline int mx_blocks(int K) { return (K + 31) / 32; }
__host__ __device__ inline int mx_stages(int K) { return (K + 255) / 256; }

// Scale factors as the tensor cores read them: chunks of 512 bytes, one for
// 128 rows x 4 blocks, row r of the 128 at (r % 32) * 16 + (r / 32) * 4 and its
// four bytes in order. Weights: [E][halves][ceil(N/128)][2 * stages][512].
size_t mx_weight_scale_bytes(int E, int halves, int N, int K);
cudaError_t launch_mx_weight_scales(const uint8_t* scales, int E, int halves, int N, int K, uint8_t* out,
                                    cudaStream_t st);

// Tensor-core product over row blocks of bn rows (mxfp4_tc.cu).
struct MxTcArgs {
  int E, N, K, gated;
  int rows;                      // rows of y
  int bn;                        // rows of a block: a multiple of 16, <= 240 (gated: <= 112)
  int nrb;                       // 128-row scale chunks of a block: ceil(bn / 128)
  int max_blocks;                // blocks the launch may find
  const int2* block_info;        // by expert: the map's (expert, rows); NULL: dense, block b = rows b * bn ...
  const int32_t* nblocks;
  const int32_t* route_of_slot;
  const uint8_t* wscale;         // launch_mx_weight_scales
  const uint8_t* xscale;         // [blocks][2 * stages][nrb][512]
  void* out;
  uint32_t* err;
  int sms;
  uint64_t wait_ns;              // limit of a pipeline wait (0: 2 s)
  int stall_issuer;              // test of the bounded waits: the issuer first waits for what never comes,
  int stall_epilogue;            // or the first epilogue warp does so for every accumulator
  CUtensorMap wmap;              // codes of W as [E * R][16 B] bytes, box 128 x 128 bytes
  CUtensorMap xmap;              // codes of x as [blocks * bn][16 B] bytes, box bn x 128 bytes
};
cudaError_t mx_weight_map(CUtensorMap* m, const uint8_t* codes, long rows, int K);
cudaError_t launch_mx_tc(MxTcArgs& a, const uint8_t* codes_x, long slots, int out_dtype, cudaStream_t st);

// Route map of the block kernel: every expert's routes in blocks of bn slots,
// in no fixed order within the expert.
struct MxMapArgs {
  const int32_t* ids;
  int R, E, bn;
  int2* block_info;        // (expert, rows) of block b, slots b * bn ...
  int32_t* nblocks;
  int32_t* route_of_slot;
  int32_t* slot_of_route;
  uint32_t* err;
};
cudaError_t launch_mx_map(const MxMapArgs& a, cudaStream_t st);

// The product for few rows in one launch (mxfp4_dec.cu): x is quantised inside
// and routes are found from the ids.
constexpr int kMxDecRows = 16;  // most rows of a chunk
struct MxDecArgs {
  int E, N, K, gated;
  int rows;             // rows of y
  int sms;
  const void* x;
  int x_dtype;
  int64_t ld;
  int vec;              // rows of x are whole eights
  const int32_t* ids;   // NULL: dense
  int topk;             // rows of y that read one row of x
  const uint8_t* wscale;
  void* out;
  int out_dtype;
  uint32_t* err;
  uint64_t wait_ns;     // as in MxTcArgs
  int stall_issuer, stall_epilogue;
  CUtensorMap wmap;
};
cudaError_t launch_mx_dec(const MxDecArgs& a, int chunks, cudaStream_t st);
// log2 of the CTAs of a cluster, among which the stages are split: as many parts
// as there are stages and SMs (two CTAs on some), at most a portable cluster.
inline int mx_dec_split(long units, int stages, int sms) {
  int l = 0;
  while (l < 3 && (2 << l) <= stages && (units << l) <= sms) ++l;
  return l;
}

// Rows of x to MXFP4 in block order: row r's codes at slot s, its scales at
// [s / bn][...][(s % bn) / 128]. dense: s = r; by expert: slot_of_route of its
// topk routes (per_route: of route r), and a route without a slot gets its row
// of `out` zeroed.
struct MxQuantArgs {
  const void* x;
  int64_t ld;
  int x_rows, K, topk;
  const int32_t* slot_of_route;  // NULL: dense
  int bn, nrb;
  uint8_t* codes;
  uint8_t* scales;
  void* out;
  int out_row_bytes;
  uint32_t* err;
};
cudaError_t launch_mx_rows_quantize(const MxQuantArgs& a, int dtype, cudaStream_t st);

}  // namespace tmoe
