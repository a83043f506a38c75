// Internal interface of the linear product and its gradient.
#pragma once

#include "common.cuh"

namespace dspark {

// out[t, f] (f contiguous, F of them) = act(lane_scale[f] col_scale[t] sum_k A[f, k] B[t, k] + bias[f]) + residual[t, f]
struct LinearArgs {
  const void* x;          // [M, K] in_type
  const void* w;          // [N, K] in_type
  const float* x_scale;   // [M] or null
  const float* w_scale;   // [N] or null
  const float* bias;      // [N] or null
  const void* residual;   // [M, N] out_type or null; may be y
  int M, N, K;
  int in_type, out_type, act;
  void* y;                // [M, N] out_type
  void* pre;              // [M, N] out_type or null
  Status* status;
};

struct LinearGradArgs {
  const void* x;          // [M, K] bf16
  const void* w;          // [N, K] bf16 (with dx)
  const void* dy;         // [M, N] bf16
  const void* pre;        // [M, N] bf16 (act != none)
  int M, N, K, act;
  void* dx;               // [M, K] bf16 or null
  void* dw;               // [N, K] bf16 or null
  float* dbias;           // [N] or null
  char* scratch;          // linear_scratch_bytes() behind the status block
  Status* status;
};

// Workspace of the backward call past the status block: dpre (with an activation)
// and partial column sums.
size_t linear_scratch_bytes(int M, int N, int act);
cudaError_t linear_launch(const LinearArgs& a, cudaStream_t s);
cudaError_t linear_grad_launch(const LinearGradArgs& a, cudaStream_t s);

}  // namespace dspark
