// C ABI of the logit head (norm, linear product) and of the token scores:
// argument checks and launches. Contracts are in include/dspark.h.
#include "host.cuh"
#include "linear.cuh"
#include "logprobs.cuh"
#include "norm.cuh"

using namespace dspark;

namespace {

// The checks every call shares: the workspace, then the device.
int ws_check(int op, int B, int K, int V, int r, int dtype, const void* ws, size_t ws_bytes, int* sms) {
  if (!ws || !aligned16(ws)) return DSPARK_ERR_INVALID_ARG;
  if (ws_bytes < dspark_workspace_bytes(op, B, K, V, r, dtype)) return DSPARK_ERR_WORKSPACE;
  return device_check(sms);
}

inline char* scratch_of(void* ws) { return static_cast<char*>(ws) + kStatusBytes; }

}  // namespace

extern "C" {

int dspark_token_logprobs(const void* logits, const int32_t* tok, const float* temp, int B, int J,
                          int V, int dtype, int n_top, float* logp, float* entropy, float* lse,
                          int32_t* top_idx, float* top_logp, void* ws, size_t ws_bytes,
                          dspark_stream_t stream) {
  if (!logits || !tok || !logp || !aligned16(logits)) return DSPARK_ERR_INVALID_ARG;
  if (!shape_ok(B, J, V, dtype)) return DSPARK_ERR_INVALID_ARG;
  if (n_top < 0 || n_top > kMaxTop || n_top > V) return DSPARK_ERR_INVALID_ARG;
  if (n_top > 0 && (!top_idx || !top_logp)) return DSPARK_ERR_INVALID_ARG;
  int sms = 0;
  if (int e = ws_check(DSPARK_OP_LOGPROBS, B, J, V, 0, dtype, ws, ws_bytes, &sms)) return e;
  LogprobArgs a;
  a.logits = logits;
  a.tok = tok;
  a.temp = temp;
  a.B = B;
  a.J = J;
  a.V = V;
  a.dtype = dtype;
  a.n_top = n_top;
  a.logp = logp;
  a.entropy = entropy;
  a.lse = lse;
  a.top_idx = top_idx;
  a.top_logp = top_logp;
  a.status = static_cast<Status*>(ws);
  return cuda_status(logprobs_launch(a, sms, (cudaStream_t)stream));
}

int dspark_token_logprobs_grad(const void* logits, const int32_t* tok, const float* temp,
                               const float* lse, const float* entropy, const float* g_logp,
                               const float* g_entropy, int B, int J, int V, int dtype,
                               void* dlogits, void* ws, size_t ws_bytes, dspark_stream_t stream) {
  if (!logits || !tok || !lse || !g_logp || !dlogits) return DSPARK_ERR_INVALID_ARG;
  if ((g_entropy != nullptr) != (entropy != nullptr)) return DSPARK_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(dlogits)) return DSPARK_ERR_INVALID_ARG;
  if (!shape_ok(B, J, V, dtype)) return DSPARK_ERR_INVALID_ARG;
  int sms = 0;
  if (int e = ws_check(DSPARK_OP_LOGPROBS, B, J, V, 0, dtype, ws, ws_bytes, &sms)) return e;
  LogprobGradArgs a;
  a.logits = logits;
  a.tok = tok;
  a.temp = temp;
  a.lse = lse;
  a.entropy = entropy;
  a.g_logp = g_logp;
  a.g_entropy = g_entropy;
  a.B = B;
  a.J = J;
  a.V = V;
  a.dtype = dtype;
  a.dlogits = dlogits;
  a.status = static_cast<Status*>(ws);
  return cuda_status(logprobs_grad_launch(a, sms, (cudaStream_t)stream));
}

int dspark_residual_norm(const void* x, const void* delta, const void* weight, int M, int H,
                         int dtype, float eps, void* sum, void* y, int y_type, float* y_scale,
                         float* rstd, void* ws, size_t ws_bytes, dspark_stream_t stream) {
  if (!x || !weight || !y) return DSPARK_ERR_INVALID_ARG;
  if (dtype != DSPARK_F32 && dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARG;
  if (y_type != dtype && y_type != DSPARK_E4M3) return DSPARK_ERR_UNSUPPORTED;
  if (y_type == DSPARK_E4M3 && !y_scale) return DSPARK_ERR_INVALID_ARG;
  if (!norm_shape_ok(M, H) || !(eps >= 0.f)) return DSPARK_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(delta) || !aligned16(weight) || !aligned16(sum) || !aligned16(y))
    return DSPARK_ERR_INVALID_ARG;
  if (int e = ws_check(DSPARK_OP_NORM, M, 0, H, 0, 0, ws, ws_bytes, nullptr)) return e;
  NormArgs a;
  a.x = x;
  a.delta = delta;
  a.weight = weight;
  a.M = M;
  a.H = H;
  a.dtype = dtype;
  a.eps = eps;
  a.sum = sum;
  a.y = y;
  a.y_type = y_type;
  a.y_scale = y_scale;
  a.rstd = rstd;
  a.status = static_cast<Status*>(ws);
  return cuda_status(norm_launch(a, (cudaStream_t)stream));
}

int dspark_residual_norm_grad(const void* s, const void* weight, const float* rstd, const void* dy,
                              const void* dsum, int M, int H, int dtype, void* dx, float* dweight,
                              void* ws, size_t ws_bytes, dspark_stream_t stream) {
  if (!s || !weight || !rstd || !dy || !dx) return DSPARK_ERR_INVALID_ARG;
  if (dtype != DSPARK_F32 && dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARG;
  if (!norm_shape_ok(M, H)) return DSPARK_ERR_INVALID_ARG;
  if (!aligned16(s) || !aligned16(weight) || !aligned16(dy) || !aligned16(dsum) || !aligned16(dx))
    return DSPARK_ERR_INVALID_ARG;
  if (int e = ws_check(DSPARK_OP_NORM, M, 0, H, 0, 0, ws, ws_bytes, nullptr)) return e;
  NormGradArgs a;
  a.s = s;
  a.weight = weight;
  a.rstd = rstd;
  a.dy = dy;
  a.dsum = dsum;
  a.M = M;
  a.H = H;
  a.dtype = dtype;
  a.dx = dx;
  a.dweight = dweight;
  a.partial = reinterpret_cast<float*>(scratch_of(ws));
  a.status = static_cast<Status*>(ws);
  return cuda_status(norm_grad_launch(a, (cudaStream_t)stream));
}

int dspark_linear(const void* x, const void* w, const float* x_scale, const float* w_scale,
                  const float* bias, const void* residual, int M, int N, int K, int in_type,
                  int out_type, int act, void* y, void* pre, void* ws, size_t ws_bytes,
                  dspark_stream_t stream) {
  if (!x || !w || !y || !aligned16(x) || !aligned16(w)) return DSPARK_ERR_INVALID_ARG;
  if (in_type != DSPARK_BF16 && in_type != DSPARK_E4M3) return DSPARK_ERR_UNSUPPORTED;
  if (out_type != DSPARK_F32 && out_type != DSPARK_BF16) return DSPARK_ERR_UNSUPPORTED;
  if (act < DSPARK_ACT_NONE || act > DSPARK_ACT_GELU) return DSPARK_ERR_INVALID_ARG;
  const bool scaled = in_type == DSPARK_E4M3;
  if ((x_scale != nullptr) != scaled || (w_scale != nullptr) != scaled) return DSPARK_ERR_INVALID_ARG;
  if (!linear_shape_ok(M, N, K, in_type)) return DSPARK_ERR_INVALID_ARG;
  const uintptr_t es = out_type == DSPARK_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(pre) | reinterpret_cast<uintptr_t>(residual)) % es)
    return DSPARK_ERR_INVALID_ARG;
  if (int e = ws_check(DSPARK_OP_LINEAR, M, 0, N, K, in_type, ws, ws_bytes, nullptr)) return e;
  LinearArgs a;
  a.x = x;
  a.w = w;
  a.x_scale = x_scale;
  a.w_scale = w_scale;
  a.bias = bias;
  a.residual = residual;
  a.M = M;
  a.N = N;
  a.K = K;
  a.in_type = in_type;
  a.out_type = out_type;
  a.act = act;
  a.y = y;
  a.pre = pre;
  a.status = static_cast<Status*>(ws);
  return cuda_status(linear_launch(a, (cudaStream_t)stream));
}

int dspark_linear_grad(const void* x, const void* w, const void* dy, const void* pre, int M, int N,
                       int K, int act, void* dx, void* dw, float* dbias, void* ws, size_t ws_bytes,
                       dspark_stream_t stream) {
  if (!dy || (dx && !w) || (dw && !x) || (!dx && !dw && !dbias)) return DSPARK_ERR_INVALID_ARG;
  if (act < DSPARK_ACT_NONE || act > DSPARK_ACT_GELU) return DSPARK_ERR_INVALID_ARG;
  if (act != DSPARK_ACT_NONE && !pre) return DSPARK_ERR_INVALID_ARG;
  if (!linear_shape_ok(M, N, K, DSPARK_BF16) || N % 8 != 0) return DSPARK_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(dy) || !aligned16(pre) || !aligned16(dx) || !aligned16(dw))
    return DSPARK_ERR_INVALID_ARG;
  if (int e = ws_check(DSPARK_OP_LINEAR, M, act == DSPARK_ACT_NONE ? 2 : 1, N, K, DSPARK_BF16, ws, ws_bytes, nullptr)) return e;
  LinearGradArgs a;
  a.x = x;
  a.w = w;
  a.dy = dy;
  a.pre = pre;
  a.M = M;
  a.N = N;
  a.K = K;
  a.act = act;
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  a.scratch = scratch_of(ws);
  a.status = static_cast<Status*>(ws);
  return cuda_status(linear_grad_launch(a, (cudaStream_t)stream));
}

}  // extern "C"
