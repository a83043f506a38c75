// Residual addition and root-mean-square norm, to the input's type or to e4m3
// with one scale per row, and its gradient.
//
//   v = x + delta, rstd = (sum v^2 / H + eps)^(-1/2), y = v rstd w
// e4m3: scale = max |y| / 448, y8 = e4m3(y / scale). max |y| = rstd max |v w|,
// so sum v^2 and max |v w| come out of one block reduction, and the row stays
// in registers between the reduction and the output: one read of x and delta,
// one write of the sum and of y.
#include <cuda_fp8.h>

#include "norm.cuh"

namespace dspark {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // smallest normal fp32: a row of zeros keeps a usable scale

template <int DT>
__device__ __forceinline__ uint4 pack16(const float* v) {
  constexpr int N = Vec16<DT>::N;
  alignas(16) typename Elem<DT>::T d[N];
#pragma unroll
  for (int e = 0; e < N; ++e) d[e] = Elem<DT>::store_round(v[e]);
  return *reinterpret_cast<const uint4*>(d);
}

// 16 bytes held in registers as they came from memory
__device__ __forceinline__ uint4 load_raw(const void* p) { return *reinterpret_cast<const uint4*>(p); }
template <int DT>
__device__ __forceinline__ void unpack16(const uint4& q, float* v) {
  Vec16<DT>::load(&q, v);
}

// N values rounded to nearest e4m3 (saturating), N bytes
template <int N>
__device__ __forceinline__ void store_e4m3(void* p, const float* v) {
  uint32_t w[N / 4];
#pragma unroll
  for (int j = 0; j < N / 4; ++j) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * j], v[4 * j + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * j + 2], v[4 * j + 3]), __NV_SATFINITE, __NV_E4M3);
    w[j] = lo | (hi << 16);
  }
  if (N == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[N / 4 - 1]);
  else
    *reinterpret_cast<uint32_t*>(p) = w[0];
}

// Sum and NaN-propagating maximum over the block (red: 2 x 32 floats).
__device__ __forceinline__ void block_sum_max(float& s, float& m, float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  if (nw == 1) return;
  if (lane == 0) {
    red[warp] = s;
    red[32 + warp] = m;
  }
  __syncthreads();
  s = lane < nw ? red[lane] : 0.f;
  m = lane < nw ? red[32 + lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
}

// One CTA per row, NV 16-byte vectors per thread.
template <int DT, bool E4M3, int NV>
__global__ void __launch_bounds__(512) norm_kernel(NormArgs a) {
  __shared__ float red[64];
  constexpr int N = Vec16<DT>::N, es = Elem<DT>::kBytes;
  const int tid = threadIdx.x, T = blockDim.x, nvec = a.H / N;
  const long long r = blockIdx.x;
  const size_t off = (size_t)r * a.H * es;
  const char* x = static_cast<const char*>(a.x) + off;
  const char* delta = a.delta ? static_cast<const char*>(a.delta) + off : nullptr;
  float v[NV][N];
  uint4 wr[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = tid + j * T;
    if (i < nvec) {
      Vec16<DT>::load(x + (size_t)i * 16, v[j]);
      wr[j] = load_raw(static_cast<const char*>(a.weight) + (size_t)i * 16);
    }
  }
  if (delta) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * T;
      if (i < nvec) {
        float d[N];
        Vec16<DT>::load(delta + (size_t)i * 16, d);
#pragma unroll
        for (int e = 0; e < N; ++e) v[j][e] += d[e];
      }
    }
  }
  float ss = 0.f, mx = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (tid + j * T < nvec) {
      float w[N];
      unpack16<DT>(wr[j], w);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        ss = fmaf(v[j][e], v[j][e], ss);
        if (E4M3) mx = max_nan(mx, fabsf(v[j][e] * w[e]));
      }
    }
  block_sum_max(ss, mx, red);
  // NaN or a sum of squares past fp32 makes the whole row NaN
  const bool bad = !(ss < INFINITY) || (E4M3 && !(mx < INFINITY));
  const float rstd = bad ? NAN : 1.f / sqrtf(ss / (float)a.H + a.eps);
  float inv = 1.f;  // 1 / scale: finite, as the scale is a normal number
  if (E4M3) {
    const float scale = bad ? NAN : fmaxf(mx * rstd / kE4m3Max, kMinScale);
    inv = 1.f / scale;
    if (tid == 0) a.y_scale[r] = scale;
  }
  if (tid == 0) {
    if (a.rstd) a.rstd[r] = rstd;
    if (bad) report(a.status, DSPARK_STATUS_BAD_ROW, (int)r);
  }
  char* sum = a.sum ? static_cast<char*>(a.sum) + off : nullptr;
  char* y = static_cast<char*>(a.y) + (E4M3 ? (size_t)r * a.H : off);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = tid + j * T;
    if (i >= nvec) continue;
    if (sum) *reinterpret_cast<uint4*>(sum + (size_t)i * 16) = pack16<DT>(v[j]);
    float o[N], w[N];
    unpack16<DT>(wr[j], w);
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = E4M3 ? v[j][e] * w[e] * rstd * inv : v[j][e] * rstd * w[e];
    if (E4M3)
      store_e4m3<N>(y + (size_t)i * N, o);
    else
      *reinterpret_cast<uint4*>(y + (size_t)i * 16) = pack16<DT>(o);
  }
}

// dx = dsum + rstd (w dy - s rstd^2 mean(w dy s)), dweight = sum over rows of
// dy s rstd. A CTA takes rows blockIdx.x, blockIdx.x + gridDim.x, ... and keeps
// its columns' dweight in registers; the CTAs' partial rows are summed in order
// by a second kernel, so the result does not depend on timing.
template <int DT, int NV>
__global__ void __launch_bounds__(512) norm_grad_kernel(NormGradArgs a) {
  __shared__ float red[64];
  constexpr int N = Vec16<DT>::N, es = Elem<DT>::kBytes;
  const int tid = threadIdx.x, T = blockDim.x, nvec = a.H / N;
  float dw[NV][N];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < N; ++e) dw[j][e] = 0.f;
  for (long long r = blockIdx.x; r < a.M; r += gridDim.x) {
    const size_t off = (size_t)r * a.H * es;
    const float rstd = a.rstd[r];
    float s[NV][N], g[NV][N];
    float dot = 0.f, unused = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * T;
      if (i >= nvec) continue;
      float w[N];
      Vec16<DT>::load(static_cast<const char*>(a.s) + off + (size_t)i * 16, s[j]);
      Vec16<DT>::load(static_cast<const char*>(a.dy) + off + (size_t)i * 16, g[j]);
      Vec16<DT>::load(static_cast<const char*>(a.weight) + (size_t)i * 16, w);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        dw[j][e] = fmaf(g[j][e] * s[j][e], rstd, dw[j][e]);
        g[j][e] *= w[e];
        dot = fmaf(g[j][e], s[j][e], dot);
      }
    }
    block_sum_max(dot, unused, red);
    const float c = rstd * rstd * (dot / (float)a.H);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * T;
      if (i >= nvec) continue;
      float d[N];
      if (a.dsum) {
        Vec16<DT>::load(static_cast<const char*>(a.dsum) + off + (size_t)i * 16, d);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) d[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) d[e] = fmaf(rstd, fmaf(-s[j][e], c, g[j][e]), d[e]);
      *reinterpret_cast<uint4*>(static_cast<char*>(a.dx) + off + (size_t)i * 16) = pack16<DT>(d);
    }
    __syncthreads();  // red is written again by the next row
  }
  if (a.dweight) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * T;
      if (i < nvec)
#pragma unroll
        for (int e = 0; e < N; ++e) a.partial[(size_t)blockIdx.x * a.H + (size_t)i * N + e] = dw[j][e];
    }
  }
}

// out[h] = sum over the G partial rows, 32 columns a CTA, 8 rows at a time
__global__ void __launch_bounds__(256) column_sums_kernel(const float* partial, int G, int H, float* out) {
  __shared__ float part[8][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int h = blockIdx.x * 32 + lane;
  float acc = 0.f;
  if (h < H)
    for (int g = row; g < G; g += 8) acc += partial[(size_t)g * H + h];
  part[row][lane] = acc;
  __syncthreads();
  if (row == 0 && h < H) {
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) t += part[q][lane];
    out[h] = t;
  }
}

// Vectors per thread: the smallest of 1, 2, 4, 8 that a block of `most` threads
// covers a row with.
inline int vecs_per_thread(int nvec, int most) {
  int nv = 1;
  while (nv < 8 && nvec > nv * most) nv *= 2;
  return nv;
}
inline int threads_for(int nvec, int nv) { return ((nvec + nv - 1) / nv + 31) / 32 * 32; }

template <int DT, bool E4M3>
cudaError_t norm_pick(const NormArgs& a, cudaStream_t s) {
  const int nvec = a.H / Vec16<DT>::N;
  const int nv = vecs_per_thread(nvec, 256);
  const int t = threads_for(nvec, nv);
  const unsigned g = (unsigned)a.M;
  switch (nv) {
    case 1: norm_kernel<DT, E4M3, 1><<<g, t, 0, s>>>(a); break;
    case 2: norm_kernel<DT, E4M3, 2><<<g, t, 0, s>>>(a); break;
    case 4: norm_kernel<DT, E4M3, 4><<<g, t, 0, s>>>(a); break;
    default: norm_kernel<DT, E4M3, 8><<<g, t, 0, s>>>(a); break;
  }
  return cudaGetLastError();
}

template <int DT>
cudaError_t norm_grad_pick(const NormGradArgs& a, cudaStream_t s) {
  const int nvec = a.H / Vec16<DT>::N;
  const int nv = vecs_per_thread(nvec, 512);
  const int t = threads_for(nvec, nv);
  const unsigned g = (unsigned)min(a.M, kNormGradBlocks);
  switch (nv) {
    case 1: norm_grad_kernel<DT, 1><<<g, t, 0, s>>>(a); break;
    case 2: norm_grad_kernel<DT, 2><<<g, t, 0, s>>>(a); break;
    case 4: norm_grad_kernel<DT, 4><<<g, t, 0, s>>>(a); break;
    default:  // rows of 4-byte entries only: 16384 of 2 bytes are 4 vectors a thread
      if constexpr (DT == DSPARK_F32) norm_grad_kernel<DT, 8><<<g, t, 0, s>>>(a);
      break;
  }
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && a.dweight) e = column_sums_launch(a.partial, (int)g, a.H, a.dweight, s);
  return e;
}

}  // namespace

cudaError_t column_sums_launch(const float* partial, int G, int H, float* out, cudaStream_t s) {
  column_sums_kernel<<<(H + 31) / 32, 256, 0, s>>>(partial, G, H, out);
  return cudaGetLastError();
}

cudaError_t norm_launch(const NormArgs& a, cudaStream_t s) {
  if (a.dtype == DSPARK_F32)
    return a.y_type == DSPARK_E4M3 ? norm_pick<DSPARK_F32, true>(a, s) : norm_pick<DSPARK_F32, false>(a, s);
  return a.y_type == DSPARK_E4M3 ? norm_pick<DSPARK_BF16, true>(a, s) : norm_pick<DSPARK_BF16, false>(a, s);
}

cudaError_t norm_grad_launch(const NormGradArgs& a, cudaStream_t s) {
  return a.dtype == DSPARK_F32 ? norm_grad_pick<DSPARK_F32>(a, s) : norm_grad_pick<DSPARK_BF16>(a, s);
}

}  // namespace dspark
