// Products by expert with 16-bit weights: what the entry points and the kernels share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace tmoe {

// Which of the three products: y = W_e x, dx = W_e^T dy, dW_e = sum dy x^T.
enum { kExForward = 0, kExGradX = 1, kExGradW = 2 };

struct ExArgs {
  int mode, dtype, out_dtype;  // tm_dtype; out_dtype: of `out`
  int T, topk, E, N, K;
  int per_route;               // x has a row a route (else a row a token)
  const void* x;               // forward, grad_w: rows of K
  int64_t ldx;
  const void* g;               // grad_x, grad_w: dy, rows of N in route order
  int64_t ldg;
  const void* w;               // forward, grad_x: [E, N, K]
  int64_t ldw, lde;            // elements between rows, and between experts
  const int32_t* order;        // routes by expert, those of no expert last
  const int32_t* offsets;      // [E + 1]
  void* out;                   // y [R, N], dx by route [R, K], or dW [E, N, K]
  uint32_t* flags;
  uint64_t wait_ns;            // limit of a wait (0: 2 s) and which one never ends: trellis_moe_experts_set_wait_test
  int stall;
};

cudaError_t launch_ex_plan(const int32_t* ids, int R, int E, int32_t* order, int32_t* offsets, uint32_t* flags,
                           cudaStream_t st);
// dx of a token: the sum of its routes' fp32 rows, in order.
cudaError_t launch_ex_sum(const float* rows, int T, int topk, int K, void* out, int dtype, cudaStream_t st);
// One of the products; some token, addresses and strides of 16 bytes.
cudaError_t launch_ex_tc(const ExArgs& a, int sms, cudaStream_t st);

}  // namespace tmoe
