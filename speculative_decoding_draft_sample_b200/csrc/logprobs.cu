// Log probabilities of given tokens with the row's entropy and its n most
// likely alternatives, and the gradient of the first two.
//
// For a row of logits l, x = l / temp: lse = ln sum exp(x), logp(v) = x_v - lse,
// H = -sum p ln p = lse - sum p x. With M = max l and z = (l - M) log2(e) / temp,
//   s = sum 2^z, t = sum z 2^z:  lse = M / temp + ln s,
//   logp(v) = (l_v - M) / temp - ln s,  H = ln s - ln(2) t / s,
// one pass with a running maximum (s and t are rescaled when it grows:
// s' = f s, t' = f (t + d s) with d = z of the old maximum, f = 2^d).
// z is formed as a difference first, so that a row masked with the type's
// lowest value (whose product with log2(e) / temp may overflow) keeps its
// meaning, and clamped at -150 (2^z flushes to zero there), so that masked
// entries add 0 * -150, not 0 * -inf.
//
// Alternatives: a thread reads a fixed column of the row's 16-byte vectors and
// knows its column's largest entry. The n largest entries of the slice all lie
// in the n columns with the largest maxima, at or above the n-th of those
// maxima, so only these columns are read a second time (n / 256 of the slice,
// out of L2) and the few entries that pass are ranked by counting. Entries are
// compared as 64-bit keys (value, then lowest index), which are unique, so
// neither ties nor the order of the list's atomics change a result.
#include <cooperative_groups.h>

#include "logprobs.cuh"

namespace dspark {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kUnroll = 4;       // 16-byte loads in flight per thread
constexpr int kMaxCluster = 8;   // CTAs that share a row
constexpr int kCand = 1024;      // candidate list; a slice with more takes the selection loop
constexpr float kFloorZ = -150.f;
constexpr float kLn2 = 0.69314718055994530942f;

// Order-preserving key of (value, index): larger value first, then lower index.
// Zero is below every key. -0 and +0 are equal.
__device__ __forceinline__ unsigned long long entry_key(float v, int idx) {
  const uint32_t u = __float_as_uint(v + 0.f);
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((unsigned long long)o << 32) | (uint32_t)~idx;
}
__device__ __forceinline__ int key_index(unsigned long long k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// Running statistics of part of a row.
struct RowStat {
  float m;    // largest logit (-inf when empty)
  float s;    // sum 2^z
  float t;    // sum z 2^z
  float chk;  // largest logit, NaN when one was NaN
};

__device__ __forceinline__ float zdiff(float v, float m, float cs) {
  return fmaxf((v - (m == -INFINITY ? 0.f : m)) * cs, kFloorZ);
}

__device__ __forceinline__ RowStat stat_merge(const RowStat& a, const RowStat& b, float cs) {
  RowStat r;
  r.m = fmaxf(a.m, b.m);
  const float da = zdiff(a.m, r.m, cs), db = zdiff(b.m, r.m, cs);
  const float fa = ex2(da), fb = ex2(db);
  r.s = fa * a.s + fb * b.s;
  r.t = fa * fmaf(da, a.s, a.t) + fb * fmaf(db, b.s, b.t);
  r.chk = max_nan(a.chk, b.chk);
  return r;
}

__device__ __forceinline__ unsigned long long block_max_key(unsigned long long k, unsigned long long* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const unsigned long long k2 = __shfl_xor_sync(0xffffffffu, k, o);
    k = k2 > k ? k2 : k;
  }
  if (lane == 0) red[warp] = k;
  __syncthreads();
  unsigned long long best = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) best = red[w] > best ? red[w] : best;
  __syncthreads();
  return best;
}

struct Shared {
  RowStat warp_stat[kThreads / 32];
  RowStat cta_stat[kMaxCluster];                     // CTA 0: every CTA's statistics
  unsigned long long lists[kMaxCluster * kMaxTop];   // CTA 0: every CTA's n largest keys
  unsigned long long keys[kThreads];                 // the columns' largest keys
  unsigned long long cand[kCand];
  unsigned long long red[kThreads / 32];
  unsigned long long thr;                            // key of the n-th column maximum (0: fewer columns)
  int sel[kMaxTop];                                  // the columns with the n largest maxima
  int nsel, ncand;
};

// The n largest keys of this CTA's slice [v0, v1) (vectors), descending, into
// list[0..n) (zeros behind the last entry).
template <int DT>
__device__ void slice_top(Shared& sh, const char* row, int v0, int v1, float mv, int mi, int n,
                          unsigned long long* list) {
  constexpr int N = Vec16<DT>::N;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned long long key = 0;
  if (v0 + tid < v1) {  // the first entry equal to the maximum, in the batch where it appeared
    for (int j = 0; j < kUnroll && !key; ++j) {
      const int i = mi + j * kThreads;
      if (i < v1) {
        float v[N];
        Vec16<DT>::load(row + (size_t)i * 16, v);
#pragma unroll
        for (int e = N - 1; e >= 0; --e)
          if (v[e] == mv) key = entry_key(v[e], i * N + e);
      }
    }
  }
  sh.keys[tid] = key;
  if (tid == 0) {
    sh.thr = 0;
    sh.nsel = 0;
    sh.ncand = 0;
  }
  if (tid < n) list[tid] = 0;
  __syncthreads();
  int rank = 0;
  for (int j = 0; j < kThreads; ++j) rank += sh.keys[j] > key;
  if (key && rank < n) {
    sh.sel[rank] = tid;
    atomicAdd(&sh.nsel, 1);
    if (rank == n - 1) sh.thr = key;
  }
  __syncthreads();
  const int nsel = sh.nsel;
  const unsigned long long thr = sh.thr;
  for (int c = warp; c < nsel; c += kThreads / 32) {
    for (int i = v0 + sh.sel[c] + lane * kThreads; i < v1; i += 32 * kThreads) {
      float v[N];
      Vec16<DT>::load(row + (size_t)i * 16, v);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const unsigned long long k = entry_key(v[e], i * N + e);
        if (k >= thr) {
          const int at = atomicAdd(&sh.ncand, 1);
          if (at < kCand) sh.cand[at] = k;
        }
      }
    }
  }
  __syncthreads();
  const int cnt = sh.ncand;
  if (cnt <= kCand) {
    for (int c = tid; c < cnt; c += kThreads) {
      const unsigned long long k = sh.cand[c];
      int r = 0;
      for (int j = 0; j < cnt && r < n; ++j) r += sh.cand[j] > k;
      if (r < n) list[r] = k;
    }
  } else {  // very many entries above the threshold: one at a time, largest first
    const int per = (v1 - v0 + kThreads - 1) / kThreads;  // vectors of a column
    unsigned long long last = ~0ull;
    for (int r = 0; r < n; ++r) {
      unsigned long long best = 0;
      for (int q = tid; q < nsel * per; q += kThreads) {
        const int i = v0 + sh.sel[q / per] + (q % per) * kThreads;
        if (i >= v1) continue;
        float v[N];
        Vec16<DT>::load(row + (size_t)i * 16, v);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const unsigned long long k = entry_key(v[e], i * N + e);
          if (k < last && k > best) best = k;
        }
      }
      last = block_max_key(best, sh.red);
      if (tid == 0) list[r] = last;
      if (!last) break;
    }
  }
  __syncthreads();
}

// A cluster of C CTAs takes a row; CTA q reads vectors [q per, (q + 1) per).
template <int DT>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(LogprobArgs a, int C) {
  __shared__ Shared sh;
  constexpr int N = Vec16<DT>::N;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long r = blockIdx.x / C;
  const int q = blockIdx.x % C;
  const int b = (int)(r / a.J);
  const int tok = a.tok[r], n = a.n_top;
  const float tau = a.temp ? a.temp[b] : 1.f;
  const bool bad_tok = tok < -1 || tok >= a.V, bad_temp = !(tau >= 0.f);
  if (tok < 0 || bad_tok || bad_temp) {  // nothing of the row is read
    if (q == 0) {
      if (tid == 0) {
        a.logp[r] = 0.f;
        if (a.entropy) a.entropy[r] = 0.f;
        if (a.lse) a.lse[r] = 0.f;
        if (bad_tok) report(a.status, DSPARK_STATUS_BAD_TOKEN, b);
        if (bad_temp && tok != -1) report(a.status, DSPARK_STATUS_BAD_TEMP, b);
      }
      if (tid < n) {
        a.top_idx[r * n + tid] = -1;
        a.top_logp[r * n + tid] = -INFINITY;
      }
    }
    return;
  }
  const float temp = tau > 0.f ? tau : 1.f;  // greedy requests are scored at temperature 1
  const float cs = fminf(kLog2e / temp, 3.0e38f);
  const char* row = static_cast<const char*>(a.logits) + r * a.V * Elem<DT>::kBytes;
  const int nvec = a.V / N, per = (nvec + C - 1) / C;
  const int v0 = q * per, v1 = min(nvec, v0 + per);

  RowStat st = {-INFINITY, 0.f, 0.f, -INFINITY};
  int mi = v0 + tid;
  for (int i = v0 + tid; i < v1; i += kUnroll * kThreads) {
    float v[kUnroll][N];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      if (i + j * kThreads < v1) {
        Vec16<DT>::load(row + (size_t)(i + j * kThreads) * 16, v[j]);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) v[j][e] = -INFINITY;
      }
    }
    float bm = v[0][0];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) bm = max_nan(bm, v[j][e]);
    st.chk = max_nan(st.chk, bm);
    if (bm > st.m) {
      const float d = zdiff(st.m, bm, cs), f = ex2(d);
      st.t = f * fmaf(d, st.s, st.t);
      st.s *= f;
      st.m = bm;
      mi = i;
    }
    const float mz = st.m == -INFINITY ? 0.f : st.m;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float z = fmaxf((v[j][e] - mz) * cs, kFloorZ);
        const float w = ex2(z);
        st.s += w;
        st.t = fmaf(w, z, st.t);
      }
  }
  const float mv = st.m;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    RowStat p;
    p.m = __shfl_xor_sync(0xffffffffu, st.m, o);
    p.s = __shfl_xor_sync(0xffffffffu, st.s, o);
    p.t = __shfl_xor_sync(0xffffffffu, st.t, o);
    p.chk = __shfl_xor_sync(0xffffffffu, st.chk, o);
    st = stat_merge(st, p, cs);
  }
  if (lane == 0) sh.warp_stat[warp] = st;
  __syncthreads();

  cg::cluster_group cluster = cg::this_cluster();
  if (C > 1) cluster.sync();  // CTA 0's shared memory exists before it is written
  Shared* root = C > 1 ? cluster.map_shared_rank(&sh, 0) : &sh;
  if (tid == 0) {
    RowStat c = sh.warp_stat[0];
    for (int w = 1; w < kThreads / 32; ++w) c = stat_merge(c, sh.warp_stat[w], cs);
    root->cta_stat[q] = c;
  }
  if (n) slice_top<DT>(sh, row, v0, v1, mv, mi, n, root->lists + q * n);
  if (C > 1) cluster.sync();
  if (q != 0) return;
  __syncthreads();

  RowStat c = sh.cta_stat[0];
  for (int w = 1; w < C; ++w) c = stat_merge(c, sh.cta_stat[w], cs);
  const bool bad = c.chk != c.chk || c.m == INFINITY || c.m == -INFINITY;
  const float ln_s = logf(c.s);
  if (tid == 0) {
    if (bad) report(a.status, DSPARK_STATUS_BAD_ROW, b);
    const float l = Elem<DT>::load(reinterpret_cast<const typename Elem<DT>::T*>(row), tok);
    a.logp[r] = bad ? 0.f : (l - c.m) / temp - ln_s;
    if (a.entropy) a.entropy[r] = bad ? 0.f : fmaxf(0.f, ln_s - kLn2 * (c.t / c.s));
    if (a.lse) a.lse[r] = bad ? 0.f : c.m / temp + ln_s;
  }
  for (int k = tid; k < C * n; k += kThreads) {
    const unsigned long long key = sh.lists[k];
    int rank = 0;
    for (int j = 0; j < C * n; ++j) rank += sh.lists[j] > key;
    if (!bad && key && rank < n) {
      a.top_idx[r * n + rank] = key_index(key);
      a.top_logp[r * n + rank] = (key_value(key) - c.m) / temp - ln_s;
    }
  }
  if (bad && tid < n) {
    a.top_idx[r * n + tid] = -1;
    a.top_logp[r * n + tid] = -INFINITY;
  }
}

// dlogits = (1 / temp) [ g_logp (1[v = tok] - p) - g_entropy p (ln p + H) ] with
// ln p = l / temp - lse: elementwise, so a read and a write of the logits. The
// sums of the forward pass come back as lse and H.
constexpr int kGradVecs = 4;                              // vectors per thread
constexpr int kGradSeg = kThreads * kGradVecs;            // vectors per work item

template <int DT>
__global__ void __launch_bounds__(kThreads) logprobs_grad_kernel(LogprobGradArgs a, int segs, long long items) {
  constexpr int N = Vec16<DT>::N;
  using T = typename Elem<DT>::T;
  const int nvec = a.V / N;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const long long r = item / segs;
    const int seg = (int)(item - r * segs);
    const int b = (int)(r / a.J);
    const int tok = a.tok[r];
    const float tau = a.temp ? a.temp[b] : 1.f;
    const float lse = a.lse[r];
    const bool bad_tok = tok < -1 || tok >= a.V, bad_temp = !(tau >= 0.f);
    const bool bad_row = !(fabsf(lse) < INFINITY);
    const bool skip = tok < 0 || bad_tok || bad_temp || bad_row;
    if (tok != -1 && skip && seg == 0 && threadIdx.x == 0)
      report(a.status, bad_tok ? DSPARK_STATUS_BAD_TOKEN : bad_temp ? DSPARK_STATUS_BAD_TEMP : DSPARK_STATUS_BAD_ROW, b);
    const float inv = 1.f / (tau > 0.f ? tau : 1.f);
    const float gl = a.g_logp[r], gh = a.g_entropy ? a.g_entropy[r] : 0.f;
    const float H = a.g_entropy ? a.entropy[r] : 0.f;
    const char* row = static_cast<const char*>(a.logits) + r * a.V * Elem<DT>::kBytes;
    char* out = static_cast<char*>(a.dlogits) + r * a.V * Elem<DT>::kBytes;
    const int i0 = seg * kGradSeg + threadIdx.x;
    float v[kGradVecs][N];
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
      const int i = i0 + j * kThreads;
      if (!skip && i < nvec) Vec16<DT>::load(row + (size_t)i * 16, v[j]);
    }
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
      const int i = i0 + j * kThreads;
      if (i >= nvec) continue;
      alignas(16) T d[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float lp = fmaxf(fmaf(v[j][e], inv, -lse), -200.f);  // exp(-200) is zero in fp32
        const float p = ex2(lp * kLog2e);
        float g = -p * (gl + gh * (lp + H));
        if (i * N + e == tok) g += gl;
        d[e] = Elem<DT>::store_round(skip ? 0.f : g * inv);
      }
      *reinterpret_cast<uint4*>(out + (size_t)i * 16) = *reinterpret_cast<const uint4*>(d);
    }
  }
}

}  // namespace

cudaError_t logprobs_launch(const LogprobArgs& a, int num_sms, cudaStream_t s) {
  const long long rows = (long long)a.B * a.J;
  const int nvec = a.V / (a.dtype == DSPARK_F32 ? 4 : 8);
  // a row is shared by as many CTAs as give each SM two, while a CTA's slice
  // keeps a vector for every thread
  int C = 1;
  while (C < kMaxCluster && rows * C < 2LL * num_sms && nvec / (2 * C) >= kThreads) C *= 2;
  auto kern = a.dtype == DSPARK_F32 ? logprobs_kernel<DSPARK_F32> : logprobs_kernel<DSPARK_BF16>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, C);
}

cudaError_t logprobs_grad_launch(const LogprobGradArgs& a, int num_sms, cudaStream_t s) {
  const long long rows = (long long)a.B * a.J;
  const int nvec = a.V / (a.dtype == DSPARK_F32 ? 4 : 8);
  const int segs = (nvec + kGradSeg - 1) / kGradSeg;
  const long long items = rows * segs;
  const unsigned grid = (unsigned)min(items, 64LL * num_sms);
  if (a.dtype == DSPARK_F32)
    logprobs_grad_kernel<DSPARK_F32><<<grid, kThreads, 0, s>>>(a, segs, items);
  else
    logprobs_grad_kernel<DSPARK_BF16><<<grid, kThreads, 0, s>>>(a, segs, items);
  return cudaGetLastError();
}

}  // namespace dspark
