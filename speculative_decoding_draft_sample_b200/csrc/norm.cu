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

// Sum and NaN-propagating maximum over the block (red: 2 x 32 floats); returns
// whether any thread's flag is set. One block barrier: the caller alternates
// between two buffers, so the next reduction's writes meet no late reader.
__device__ __forceinline__ bool block_sum_max(float& s, float& m, float* red, bool flag) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  if (lane == 0) {
    red[warp] = s;
    red[32 + warp] = m;
  }
  const bool any = __syncthreads_or(flag);
  s = lane < nw ? red[lane] : 0.f;
  m = lane < nw ? red[32 + lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  return any;
}

// sum v^2 and max |v w| of a vector added to ss and mx
template <int DT, bool E4M3>
__device__ __forceinline__ void add_row(const float* v, const uint4& wr, float& ss, float& mx) {
  constexpr int N = Vec16<DT>::N;
  float w[N];
  if (E4M3) unpack16<DT>(wr, w);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    ss = fmaf(v[e], v[e], ss);
    if (E4M3) mx = max_nan(mx, fabsf(v[e] * w[e]));
  }
}

// (rstd, 1 / scale) of row r from its sums; one thread writes them out.
template <bool E4M3>
__device__ __forceinline__ float2 row_factors(const NormArgs& a, long long r, float ss, float mx, bool one) {
  // NaN or a sum of squares past fp32 makes the whole row NaN
  const bool bad = !(ss < INFINITY) || (E4M3 && !(mx < INFINITY));
  const float rstd = bad ? NAN : 1.f / sqrtf(ss / (float)a.H + a.eps);
  float inv = 1.f;  // 1 / scale: finite, as the scale is a normal number
  if (E4M3) {
    const float scale = bad ? NAN : fmaxf(mx * rstd / kE4m3Max, kMinScale);
    inv = 1.f / scale;
    if (one) a.y_scale[r] = scale;
  }
  if (one) {
    if (a.rstd) a.rstd[r] = rstd;
    if (bad) report(a.status, DSPARK_STATUS_BAD_ROW, (int)r);
  }
  return make_float2(rstd, inv);
}

// Vector i of row r: the sum and y. e4m3: v w times rstd and 1 / scale, two rounded fp32
// factors where the definition divides once; 2^-23 of the value, so an entry next to a tie
// of e4m3 may fall on its other side.
template <int DT, bool E4M3>
__device__ __forceinline__ void write_row(const NormArgs& a, long long r, int i, const float* v, const uint4& wr, float2 k) {
  constexpr int N = Vec16<DT>::N, es = Elem<DT>::kBytes;
  const size_t off = (size_t)r * a.H * es + (size_t)i * 16;
  if (a.sum) *reinterpret_cast<uint4*>(static_cast<char*>(a.sum) + off) = pack16<DT>(v);
  float o[N], w[N];
  unpack16<DT>(wr, w);
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = E4M3 ? v[e] * w[e] * k.x * k.y : v[e] * k.x * w[e];
  if (E4M3)
    store_e4m3<N>(static_cast<char*>(a.y) + (size_t)r * a.H + (size_t)i * N, o);
  else
    *reinterpret_cast<uint4*>(static_cast<char*>(a.y) + off) = pack16<DT>(o);
}

// A vector's share of dweight and of sum w dy s.
template <int DT>
__device__ __forceinline__ void add_grad(const uint4& sr, const uint4& gr, const float* w, float rstd, float* dw, float& dot) {
  constexpr int N = Vec16<DT>::N;
  float s[N], g[N];
  unpack16<DT>(sr, s);
  unpack16<DT>(gr, g);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float gs = g[e] * s[e];
    dw[e] = fmaf(gs, rstd, dw[e]);
    dot = fmaf(gs, w[e], dot);
  }
}

// dx of a vector; c = rstd^2 mean(w dy s)
template <int DT>
__device__ __forceinline__ uint4 grad16(const uint4& sr, const uint4& gr, const uint4& dr, const float* w, float rstd, float c) {
  constexpr int N = Vec16<DT>::N;
  float s[N], g[N], d[N];
  unpack16<DT>(sr, s);
  unpack16<DT>(gr, g);
  unpack16<DT>(dr, d);
#pragma unroll
  for (int e = 0; e < N; ++e) d[e] = fmaf(rstd, fmaf(-s[e], c, g[e] * w[e]), d[e]);
  return pack16<DT>(d);
}

enum : unsigned int { kWhereNormRow = 60 };  // wait site recorded when a bounded wait gives up

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

constexpr int kMaxStages = 4;

// The rows blockIdx.x, blockIdx.x + gridDim.x, ... of up to three matrices, fed
// through a ring of `stages` shared-memory rows. Row number it is read between
// wait(it) and refill(it), the latter by every thread after a block barrier that
// follows the reads.
template <int ARRAYS>
struct RowFeed {
  unsigned char* ring;
  unsigned long long* full;
  const char* src[ARRAYS];
  int stages, bytes, rows;

  __device__ __forceinline__ void issue(int it) const {
    const long long r = blockIdx.x + (long long)it * gridDim.x;
    if (r >= rows) return;
    const int st = it % stages;
    int n = 0;
#pragma unroll
    for (int k = 0; k < ARRAYS; ++k) n += src[k] != nullptr;
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(full + st)), "r"(n * bytes) : "memory");
#pragma unroll
    for (int k = 0; k < ARRAYS; ++k)
      if (src[k])
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                saddr(ring + (size_t)(st * ARRAYS + k) * bytes)),
            "l"(src[k] + r * bytes), "r"(bytes), "r"(saddr(full + st))
            : "memory");
  }
  __device__ __forceinline__ void start() const {
    if (threadIdx.x == 0) {
      for (int i = 0; i < stages; ++i)
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(saddr(full + i)) : "memory");
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    grid_wait();
    if (threadIdx.x == 0) {
      for (int i = 0; i < stages; ++i) issue(i);
    }
    __syncthreads();
  }
  __device__ __forceinline__ bool wait(int it) const {
    return mbar_wait_bounded(saddr(full + it % stages), (it / stages) & 1);
  }
  __device__ __forceinline__ const unsigned char* row(int it, int k) const {
    return ring + (size_t)(it % stages * ARRAYS + k) * bytes;
  }
  __device__ __forceinline__ void refill(int it) const {
    if (threadIdx.x == 0) issue(it + stages);
  }
  // after a wait for row `it` gave up: let the copies on their way land
  __device__ __forceinline__ void drain(int it) const {
    if (threadIdx.x == 0)
      for (int i = it; i < it + stages; ++i)
        if (blockIdx.x + (long long)i * gridDim.x < rows) wait(i);
  }
};

// NV 16-byte vectors of a row per thread.
template <int DT, bool E4M3, int NV>
__global__ void __launch_bounds__(512, NV <= 2 ? 2 : 1) norm_kernel(NormArgs a, int stages) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ unsigned long long full[kMaxStages];
  __shared__ float red[2][64];
  constexpr int N = Vec16<DT>::N, es = Elem<DT>::kBytes;
  const int tid = threadIdx.x, T = blockDim.x, nvec = a.H / N;
  const RowFeed<2> feed = {ring, full, {static_cast<const char*>(a.x), static_cast<const char*>(a.delta)}, stages, a.H * es, a.M};
  feed.start();
  uint4 wr[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (tid + j * T < nvec) wr[j] = load_raw(static_cast<const char*>(a.weight) + (size_t)(tid + j * T) * 16);
  int it = 0;
  for (long long r = blockIdx.x; r < a.M; r += gridDim.x, ++it) {
    const bool arrived = feed.wait(it);
    float v[NV][N];
    float ss = 0.f, mx = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * T;
      if (i >= nvec) continue;
      Vec16<DT>::load(feed.row(it, 0) + i * 16, v[j]);
      if (a.delta) {
        float d[N];
        Vec16<DT>::load(feed.row(it, 1) + i * 16, d);
#pragma unroll
        for (int e = 0; e < N; ++e) v[j][e] += d[e];
      }
      add_row<DT, E4M3>(v[j], wr[j], ss, mx);
    }
    if (block_sum_max(ss, mx, red[it & 1], !arrived)) {  // a wait gave up
      feed.drain(it);
      if (tid == 0) report_wait(a.status, kWhereNormRow, (int)r);
      return;
    }
    feed.refill(it);
    const float2 k = row_factors<E4M3>(a, r, ss, mx, tid == 0);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (tid + j * T < nvec) write_row<DT, E4M3>(a, r, tid + j * T, v[j], wr[j], k);
  }
}

// dx = dsum + rstd (w dy - s rstd^2 mean(w dy s)), dweight = sum over rows of
// dy s rstd. A CTA's rows come as above; it keeps its columns' dweight in
// registers, and the CTAs' partial rows are summed in order by a second kernel, so
// the result does not depend on timing.
template <int DT, int NV>
__global__ void __launch_bounds__(512, NV == 1 ? 2 : 1) norm_grad_kernel(NormGradArgs a, int stages) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ unsigned long long full[kMaxStages];
  __shared__ float red[2][64];
  constexpr int N = Vec16<DT>::N, es = Elem<DT>::kBytes;
  const int tid = threadIdx.x, T = blockDim.x, nvec = a.H / N;
  const RowFeed<3> feed = {ring, full,
                           {static_cast<const char*>(a.s), static_cast<const char*>(a.dy), static_cast<const char*>(a.dsum)},
                           stages, a.H * es, a.M};
  grid_release();
  feed.start();
  constexpr bool kKeep = NV * N <= 16;  // weights in registers (else read again, out of L2)
  float dw[NV][N];
  uint4 wr[kKeep ? NV : 1] = {};
  auto weights = [&](int j, float* w) {
    unpack16<DT>(kKeep ? wr[kKeep ? j : 0] : load_raw(static_cast<const char*>(a.weight) + (size_t)(tid + j * T) * 16), w);
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (kKeep && tid + j * T < nvec) wr[kKeep ? j : 0] = load_raw(static_cast<const char*>(a.weight) + (size_t)(tid + j * T) * 16);
#pragma unroll
    for (int e = 0; e < N; ++e) dw[j][e] = 0.f;
  }
  int it = 0;
  for (long long r = blockIdx.x; r < a.M; r += gridDim.x, ++it) {
    const size_t off = (size_t)r * a.H * es;
    const float rstd = a.rstd[r];  // an ordinary load: the launch before may have written it
    const bool arrived = feed.wait(it);
    uint4 sr[NV], gr[NV], dr[NV];
    float dot = 0.f, unused = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * T;
      if (i >= nvec) continue;
      sr[j] = load_raw(feed.row(it, 0) + i * 16);
      gr[j] = load_raw(feed.row(it, 1) + i * 16);
      dr[j] = a.dsum ? load_raw(feed.row(it, 2) + i * 16) : make_uint4(0, 0, 0, 0);
      float w[N];
      weights(j, w);
      add_grad<DT>(sr[j], gr[j], w, rstd, dw[j], dot);
    }
    if (block_sum_max(dot, unused, red[it & 1], !arrived)) {  // a wait gave up
      feed.drain(it);
      if (tid == 0) report_wait(a.status, kWhereNormRow, (int)r);
      return;
    }
    feed.refill(it);
    const float c = rstd * rstd * (dot / (float)a.H);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * T;
      if (i >= nvec) continue;
      float w[N];
      weights(j, w);
      *reinterpret_cast<uint4*>(static_cast<char*>(a.dx) + off + (size_t)i * 16) = grad16<DT>(sr[j], gr[j], dr[j], w, rstd, c);
    }
  }
  if (a.dweight) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * T;
      if (i < nvec) {
        float4* p = reinterpret_cast<float4*>(a.partial + (size_t)blockIdx.x * a.H + (size_t)i * N);
#pragma unroll
        for (int e = 0; e < N; e += 4) p[e / 4] = make_float4(dw[j][e], dw[j][e + 1], dw[j][e + 2], dw[j][e + 3]);
      }
    }
  }
}

// Narrow rows (up to 128 16-byte vectors): a warp per row, NV vectors a lane, no
// barrier and no ring; many warps keep memory busy. With a CTA per row the gradient
// of m8039 h272 took 29 us, most of it barriers.
constexpr int kRowWarps = 8;

__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <int DT, bool E4M3, int NV>
__global__ void __launch_bounds__(32 * kRowWarps) norm_rows_kernel(NormArgs a) {
  grid_wait();
  constexpr int N = Vec16<DT>::N, es = Elem<DT>::kBytes;
  const int lane = threadIdx.x & 31, nvec = a.H / N;
  for (long long r = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5); r < a.M; r += (long long)gridDim.x * kRowWarps) {
    const size_t off = (size_t)r * a.H * es;
    float v[NV][N];
    uint4 wr[NV], dr[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = lane + j * 32;
      if (i >= nvec) continue;
      Vec16<DT>::load(static_cast<const char*>(a.x) + off + (size_t)i * 16, v[j]);
      if (a.delta) dr[j] = load_raw(static_cast<const char*>(a.delta) + off + (size_t)i * 16);
      wr[j] = load_raw(static_cast<const char*>(a.weight) + (size_t)i * 16);
    }
    float ss = 0.f, mx = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (lane + j * 32 >= nvec) continue;
      if (a.delta) {
        float d[N];
        unpack16<DT>(dr[j], d);
#pragma unroll
        for (int e = 0; e < N; ++e) v[j][e] += d[e];
      }
      add_row<DT, E4M3>(v[j], wr[j], ss, mx);
    }
    ss = warp_sum(ss);
    if (E4M3) mx = warp_max_nan(mx);
    const float2 k = row_factors<E4M3>(a, r, ss, mx, lane == 0);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (lane + j * 32 < nvec) write_row<DT, E4M3>(a, r, lane + j * 32, v[j], wr[j], k);
  }
}

template <int DT, int NV>
__global__ void __launch_bounds__(32 * kRowWarps) norm_grad_rows_kernel(NormGradArgs a) {
  constexpr int N = Vec16<DT>::N, es = Elem<DT>::kBytes;
  __shared__ float sums[kRowWarps][NV * 32 * N];
  grid_release();
  grid_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nvec = a.H / N;
  float dw[NV][N];
  uint4 wr[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (lane + j * 32 < nvec) wr[j] = load_raw(static_cast<const char*>(a.weight) + (size_t)(lane + j * 32) * 16);
#pragma unroll
    for (int e = 0; e < N; ++e) dw[j][e] = 0.f;
  }
  for (long long r = (long long)blockIdx.x * kRowWarps + warp; r < a.M; r += (long long)gridDim.x * kRowWarps) {
    const size_t off = (size_t)r * a.H * es;
    const float rstd = a.rstd[r];  // an ordinary load: the launch before may have written it
    uint4 sr[NV], gr[NV], dr[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = lane + j * 32;
      if (i >= nvec) continue;
      sr[j] = load_raw(static_cast<const char*>(a.s) + off + (size_t)i * 16);
      gr[j] = load_raw(static_cast<const char*>(a.dy) + off + (size_t)i * 16);
      dr[j] = a.dsum ? load_raw(static_cast<const char*>(a.dsum) + off + (size_t)i * 16) : make_uint4(0, 0, 0, 0);
    }
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (lane + j * 32 >= nvec) continue;
      float w[N];
      unpack16<DT>(wr[j], w);
      add_grad<DT>(sr[j], gr[j], w, rstd, dw[j], dot);
    }
    dot = warp_sum(dot);
    const float c = rstd * rstd * (dot / (float)a.H);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = lane + j * 32;
      if (i >= nvec) continue;
      float w[N];
      unpack16<DT>(wr[j], w);
      *reinterpret_cast<uint4*>(static_cast<char*>(a.dx) + off + (size_t)i * 16) = grad16<DT>(sr[j], gr[j], dr[j], w, rstd, c);
    }
  }
  if (!a.dweight) return;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < N; ++e) sums[warp][(lane + j * 32) * N + e] = dw[j][e];
  __syncthreads();
  for (int h = threadIdx.x; h < a.H; h += 32 * kRowWarps) {
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < kRowWarps; ++q) t += sums[q][h];
    a.partial[(size_t)blockIdx.x * a.H + h] = t;
  }
}

// out[h] = sum over the G partial rows: 32 columns a CTA, a warp every 32nd row,
// four of them in flight (a warp every eighth row one at a time took 7 us for 296
// rows of 4096, more than twice as long).
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* partial, int G, int H, float* out, int order) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int h = blockIdx.x * 32 + lane;
  float acc = 0.f;
  if (order == kAfter) grid_wait();
  if (h < H) {
    for (int g = row; g < G; g += 128) {
      float d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = g + 32 * j < G ? __ldcg(partial + (size_t)(g + 32 * j) * H + h) : 0.f;
      acc += (d[0] + d[1]) + (d[2] + d[3]);
    }
  }
  part[row][lane] = acc;
  __syncthreads();
  const float t = warp_sum(part[lane][row]);
  if (lane == 0 && blockIdx.x * 32 + row < H) out[blockIdx.x * 32 + row] = t;
  if (order == kBeside) grid_wait();
}

// Shared memory that the rings of an SM's blocks have together.
constexpr int kRing = 216 * 1024;

// How a call's rows are cut: threads of a block and vectors per thread (the fewest
// of 1, 2, 4, 8 that 512 threads cover a row with), blocks per SM, and the ring's
// depth (up to 4 rows within the SM's shared memory).
struct Cut {
  int nv, threads, blocks, stages, smem;
};
inline Cut make_cut(int M, int H, int dtype, int arrays, int most_blocks) {
  const int es = dtype == DSPARK_F32 ? 4 : 2, nvec = H * es / 16, row = arrays * H * es;
  Cut c;
  c.nv = 1;
  while (c.nv < 8 && nvec > c.nv * 512) c.nv *= 2;
  c.threads = ((nvec + c.nv - 1) / c.nv + 31) / 32 * 32;
  int per_sm = c.nv > most_blocks ? 1 : (c.threads > 256 ? 2 : 4);
  while (per_sm > 1 && kRing / per_sm < 2 * row) per_sm /= 2;
  c.stages = max(1, min(kMaxStages, kRing / per_sm / row));
  c.smem = c.stages * row;
  c.blocks = min(M, 148 * per_sm);
  return c;
}

// The kernel's limit is the largest ring of any call, the same in every call: it belongs
// to the kernel on its device, and a call of another host thread may set it between this
// call's setting and its launch.
template <typename Kern, typename Args>
cudaError_t launch(Kern kern, const Args& a, const Cut& c, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing);
  if (e != cudaSuccess) return e;
  return launch_early(kern, c.blocks, c.threads, c.smem, 1, s, a, c.stages);
}

// Rows of up to 128 vectors: enough CTAs of 8 rows for eight on every SM.
inline int row_blocks(int M, int most) { return min((M - 1) / kRowWarps + 1, most); }  // (M may be INT_MAX)

template <int DT, bool E4M3>
cudaError_t norm_pick(const NormArgs& a, cudaStream_t s) {
  const int nvec = a.H / Vec16<DT>::N;
  if (nvec <= 128) {
    auto kern = nvec <= 32 ? norm_rows_kernel<DT, E4M3, 1> : nvec <= 64 ? norm_rows_kernel<DT, E4M3, 2> : norm_rows_kernel<DT, E4M3, 4>;
    return launch_early(kern, row_blocks(a.M, 8 * 148), 32 * kRowWarps, 0, 1, s, a);
  }
  const Cut c = make_cut(a.M, a.H, DT, 2, 2);
  switch (c.nv) {
    case 1: return launch(norm_kernel<DT, E4M3, 1>, a, c, s);
    case 2: return launch(norm_kernel<DT, E4M3, 2>, a, c, s);
    case 4: return launch(norm_kernel<DT, E4M3, 4>, a, c, s);
    default:  // rows of 4-byte entries only: 16384 of 2 bytes are 4 vectors a thread
      if constexpr (DT == DSPARK_F32) return launch(norm_kernel<DT, E4M3, 8>, a, c, s);
      return cudaErrorInvalidValue;
  }
}

template <int DT>
cudaError_t norm_grad_pick(const NormGradArgs& a, cudaStream_t s) {
  Cut c = make_cut(a.M, a.H, DT, 3, 1);
  c.blocks = min(c.blocks, kNormGradBlocks);
  NormGradArgs b = a;
  cudaError_t e;
  const int nvec = a.H / Vec16<DT>::N;
  if (nvec <= 128) {
    c.blocks = row_blocks(a.M, kNormGradBlocks);
    if (c.blocks == 1) b.partial = a.dweight;  // one CTA's sums are the result
    auto kern = nvec <= 32 ? norm_grad_rows_kernel<DT, 1> : nvec <= 64 ? norm_grad_rows_kernel<DT, 2> : norm_grad_rows_kernel<DT, 4>;
    e = launch_early(kern, c.blocks, 32 * kRowWarps, 0, 1, s, b);
    if (e == cudaSuccess && a.dweight && c.blocks > 1) e = column_sums_launch(a.partial, c.blocks, a.H, a.dweight, s, kAfter);
    return e;
  }
  // (dweight may be aligned to 4 bytes only, the wide kernels store 16 at a time)
  if (c.blocks == 1 && (reinterpret_cast<uintptr_t>(a.dweight) & 15) == 0) b.partial = a.dweight;
  switch (c.nv) {
    case 1: e = launch(norm_grad_kernel<DT, 1>, b, c, s); break;
    case 2: e = launch(norm_grad_kernel<DT, 2>, b, c, s); break;
    case 4: e = launch(norm_grad_kernel<DT, 4>, b, c, s); break;
    default:
      if constexpr (DT == DSPARK_F32)
        e = launch(norm_grad_kernel<DT, 8>, b, c, s);
      else
        e = cudaErrorInvalidValue;
  }
  if (e == cudaSuccess && a.dweight && b.partial != a.dweight) e = column_sums_launch(a.partial, c.blocks, a.H, a.dweight, s, kAfter);
  return e;
}

}  // namespace

cudaError_t column_sums_launch(const float* partial, int G, int H, float* out, cudaStream_t s, Order order) {
  return launch_early(column_sums_kernel, dim3((H + 31) / 32), 1024, 0, 1, s, partial, G, H, out, (int)order);
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
