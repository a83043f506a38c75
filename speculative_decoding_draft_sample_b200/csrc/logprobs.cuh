// Internal interface of the token log-probability kernels.
#pragma once

#include "common.cuh"

namespace dspark {

constexpr int kMaxTop = 32;  // most alternatives a call returns

struct LogprobArgs {
  const void* logits;       // [B, J, V]
  const int32_t* tok;       // [B, J], -1 = padding
  const float* temp;        // [B] or null (1)
  int B, J, V, dtype;
  int n_top;
  float* logp;              // [B, J]
  float* entropy;           // [B, J] or null
  float* lse;               // [B, J] or null
  int32_t* top_idx;         // [B, J, n_top] (n_top > 0)
  float* top_logp;          // [B, J, n_top] (n_top > 0)
  Status* status;
};

struct LogprobGradArgs {
  const void* logits;       // [B, J, V]
  const int32_t* tok;       // [B, J]
  const float* temp;        // [B] or null
  const float* lse;         // [B, J]
  const float* entropy;     // [B, J] (with g_entropy)
  const float* g_logp;      // [B, J]
  const float* g_entropy;   // [B, J] or null
  int B, J, V, dtype;
  void* dlogits;            // [B, J, V]
  Status* status;
};

cudaError_t logprobs_launch(const LogprobArgs& a, int num_sms, cudaStream_t s);
cudaError_t logprobs_grad_launch(const LogprobGradArgs& a, int num_sms, cudaStream_t s);

}  // namespace dspark
