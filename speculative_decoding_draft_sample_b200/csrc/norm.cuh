// Internal interface of the residual-norm kernels.
#pragma once

#include "common.cuh"
#include "launch.cuh"

namespace dspark {

struct NormArgs {
  const void* x;        // [M, H]
  const void* delta;    // [M, H] or null
  const void* weight;   // [H]
  int M, H, dtype;
  float eps;
  void* sum;            // [M, H] or null; may be x or delta
  void* y;              // [M, H] of y_type
  int y_type;           // the input's dtype or DSPARK_E4M3
  float* y_scale;       // [M] (DSPARK_E4M3)
  float* rstd;          // [M] or null
  Status* status;
};

struct NormGradArgs {
  const void* s;        // [M, H] the normalised sums
  const void* weight;   // [H]
  const float* rstd;    // [M]
  const void* dy;       // [M, H]
  const void* dsum;     // [M, H] or null
  int M, H, dtype;
  void* dx;             // [M, H]; may be dy or dsum
  float* dweight;       // [H] or null
  float* partial;       // [kNormGradBlocks, H] (workspace)
  Status* status;
};

// Most CTAs of the backward pass, one partial row of dweight each (two for each of 148 SMs)
constexpr int kNormGradBlocks = 296;

cudaError_t norm_launch(const NormArgs& a, cudaStream_t s);
cudaError_t norm_grad_launch(const NormGradArgs& a, cudaStream_t s);

// out[h] = sum over g < G of partial[g, h], in a fixed order.
cudaError_t column_sums_launch(const float* partial, int G, int H, float* out, cudaStream_t s, Order order);

}  // namespace dspark
