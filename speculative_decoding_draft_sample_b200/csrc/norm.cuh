// Internal interface of the residual-norm kernels.
#pragma once

#include "common.cuh"

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

// A launch that may start while the one before it in the stream still runs: kBeside
// shares no output with it and no input that either writes, and waits for it before it
// ends; kAfter reads what it wrote, and waits for it before its
// first load of that.
enum : int { kAlone, kBeside, kAfter };

// out[h] = sum over g < G of partial[g, h], in a fixed order; order is kBeside or kAfter
// (m8192 h4096 with the launch before: 52.4 us kAfter, 55.5 as a plain launch).
cudaError_t column_sums_launch(const float* partial, int G, int H, float* out, cudaStream_t s, int order);

}  // namespace dspark
