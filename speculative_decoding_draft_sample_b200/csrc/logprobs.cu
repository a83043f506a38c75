// Log probabilities of given tokens with the row's entropy and its n most
// likely alternatives, and the gradient of the first two.
//
// For a row of logits l, x = l / temp: lse = ln sum exp(x), logp(v) = x_v - lse,
// H = -sum p ln p = lse - sum p x. With M = max l and z = (l - M) log2(e) / temp,
//   s = sum 2^z, t = sum z 2^z:  lse = M / temp + ln s,
//   logp(v) = (l_v - M) / temp - ln s,  H = ln s - ln(2) t / s,
// one pass with a running maximum (s and t are rescaled when it grows:
// s' = f s, t' = f (t + d s) with d = z of the old maximum, f = 2^d).
//
// The pass is bound by instructions before it is bound by memory (bf16: 22
// entries a nanosecond and SM at the copy rate), so an entry costs about five:
// maxima and the clamp below on packed bf16 pairs, differences, products and sums
// on packed fp32 pairs, one 2^z. z = l cs - round(M cs) is one fused product (cs =
// log2(e) / temp); the rounding of M cs is known and taken out of the thread's sums
// at the end. It is at most 1/4 there: a thread whose own maximum has |M cs| >= 2^23
// (a column of masked entries, of whatever value) adds nothing, and where the row's
// maximum has |M cs| >= 2^22, so that such a thread might count, a plain second pass
// takes differences before it scales them. Logits are clamped at M - 200 / cs,
// rounded down: 2^z is zero there, and masked entries (-inf or any finite value) add
// 0 * finite, never 0 * inf.
//
// Alternatives: a thread reads a fixed column of the row's 16-byte vectors and
// knows its column's largest entry. The n largest entries of the slice all lie
// in the columns with the n largest maxima, at or above the n-th of those maxima.
// One warp finds a value that n to n + 8 maxima reach by bisection; of these
// columns the segments (up to 8 in a column) whose own maxima reach it are read a
// second time, out of L2, and the few entries that pass are ranked by counting.
// Where equal maxima leave more than n + 8 columns, they are chosen by 64-bit keys
// (value, then lowest index). Candidates are always ranked
// by these keys, which are unique, so neither ties nor the order of the list's
// atomics change a result.
//
// Measured: b256 j6 v129280 with 42 % of the rows padded away and 5 alternatives 56 us
// (4.1 TB/s; 51 without alternatives, 46 with neither exponentials nor alternatives);
// b64 j6 v151936 in fp32 without alternatives 40 us (5.8 TB/s).
#include <climits>

#include <cooperative_groups.h>

#include "launch.cuh"
#include "logprobs.cuh"

namespace dspark {

namespace {

namespace cg = cooperative_groups;

enum : unsigned int {  // wait sites recorded when a bounded wait gives up
  kWhereEmpty = 50,
  kWhereFull = 51,
};

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

constexpr int kThreads = 256;      // readers; one more warp feeds them
constexpr int kUnroll = 4;       // 16-byte vectors of a thread in a ring slot
constexpr int kSlotVecs = kUnroll * kThreads;
constexpr int kSlots = 2;        // ring of 16 KB slots: with four CTAs on an SM up to 128 KB are on their way
constexpr int kCtasPerSm = 4;
constexpr int kMaxCluster = 8;   // CTAs that share a row
constexpr int kCand = 1024;      // candidate list; a slice with more takes the selection loop
constexpr int kSegs = 8;         // segments of a column with a maximum of their own, at most
constexpr int kUnits = 256;      // list of segments to read again; where it is full, whole columns are read
constexpr int kSlack = 8;        // columns that the bisection may take beyond n
constexpr float kFloorZ = -150.f;
constexpr float kClampZ = 200.f;
constexpr float kFarZ = 8388608.f;    // 2^23: a thread's maximum past this z adds nothing (rounding of z below: 1/4)
constexpr float kPlainZ = 4194304.f;  // 2^22: a row's maximum past this z takes the plain pass
constexpr float kMaxTemp = 1.0e30f;   // past this a temperature is an error
constexpr float kLn2 = 0.69314718055994530942f;

// Order-preserving key of (value, index): larger value first, then lower index.
// Zero is below every key. -0 and +0 are equal.
__device__ __forceinline__ uint32_t value_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ unsigned long long entry_key(float v, int idx) {
  return ((unsigned long long)value_key(v) << 32) | (uint32_t)~idx;
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

// Barrier of the eight reading warps.
__device__ __forceinline__ void readers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

__device__ __forceinline__ unsigned long long block_max_key(unsigned long long k, unsigned long long* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const unsigned long long k2 = __shfl_xor_sync(0xffffffffu, k, o);
    k = k2 > k ? k2 : k;
  }
  if (lane == 0) red[warp] = k;
  readers_sync();
  unsigned long long best = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) best = red[w] > best ? red[w] : best;
  readers_sync();
  return best;
}

// Two fp32 values in one 64-bit register pair, and arithmetic on both at once.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A 16-byte vector as four 32-bit words: two bf16 entries or one fp32 entry each.
template <int DT>
struct Words;
template <>
struct Words<DSPARK_BF16> {
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  __device__ __forceinline__ static uint32_t max_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ __forceinline__ static uint32_t max_num(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ __forceinline__ static float top(uint32_t w) {
    return dspark::max_nan(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  // the largest value of the type not above v, in both halves (finite)
  __device__ __forceinline__ static uint32_t floor_of(float v) {
    const uint32_t u = __float_as_uint(v);
    uint32_t h = u >> 16;
    if ((u & 0x80000000u) && (u & 0xffffu)) ++h;
    if (h > 0xff7fu) h = 0xff7fu;
    return h | (h << 16);
  }
  // the entry pairs of a vector
  __device__ __forceinline__ static f32x2 pair(const uint32_t* w, int i) {
    return pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
};
template <>
struct Words<DSPARK_F32> {
  static constexpr uint32_t kNegInf = 0xff800000u;
  __device__ __forceinline__ static uint32_t max_nan(uint32_t a, uint32_t b) {
    return __float_as_uint(dspark::max_nan(__uint_as_float(a), __uint_as_float(b)));
  }
  __device__ __forceinline__ static uint32_t max_num(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
  __device__ __forceinline__ static float top(uint32_t w) { return __uint_as_float(w); }
  __device__ __forceinline__ static uint32_t floor_of(float v) { return __float_as_uint(fmaxf(v, -3.4028234663852886e38f)); }
  __device__ __forceinline__ static f32x2 pair(const uint32_t* w, int i) {
    return pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
};

struct Shared {
  uint4 ring[kSlots][kSlotVecs];
  unsigned long long full[kSlots], empty[kSlots];    // mbarriers
  RowStat warp_stat[kThreads / 32];
  RowStat cta_stat[kMaxCluster];                     // CTA 0: every CTA's statistics
  unsigned long long lists[kMaxCluster * kMaxTop];   // CTA 0: every CTA's n largest keys
  uint32_t vals[kThreads];                           // the columns' largest values (value_key), 0 = no entry
  float seg_max[kSegs][kThreads];                    // the columns' segments' largest values
  unsigned long long keys[kThreads];                 // the same as full keys, where values tie
  unsigned long long cand[kCand];
  unsigned long long red[kThreads / 32];
  unsigned long long thr;                            // the bound
  int sel[kMaxTop + kSlack];                         // the columns that reach it
  int nsel, ncand;
  int units[kUnits];                                 // (segment, column) pairs to read again
  int nunit;
  int ties;                                          // equal maxima left too many columns
  int dead;                                          // a bounded wait gave up
};

// By one warp: a bound that at least n and at most n + kSlack of 256 keys reach
// (all nonzero ones when there are no more than that); false when equal keys make
// that impossible.
template <typename Key>
__device__ __forceinline__ bool bisect(const Key* keys, int n, int lane, Key lo, Key hi, Key* bound) {
  constexpr int kPer = kThreads / 32;
  Key k[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) k[j] = keys[j * 32 + lane];
  auto reach = [&](Key b) {
    int c = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) c += k[j] >= b;
    return (int)__reduce_add_sync(0xffffffffu, c);
  };
  int c = reach(lo);  // invariant: at least n reach lo (or all do), fewer than n reach hi + 1
  while (c > n + kSlack && lo < hi) {
    const Key mid = lo + (hi - lo) / 2 + 1;  // lo < mid <= hi
    const int cm = reach(mid);
    if (cm >= n) {
      lo = mid;
      c = cm;
    } else {
      hi = mid - 1;
    }
  }
  *bound = lo;
  return c <= n + kSlack;
}

// The columns whose key reaches the bound.
template <typename Key>
__device__ __forceinline__ void list_columns(Shared& sh, const Key* keys, Key bound, int lane) {
  int at = 0;
#pragma unroll
  for (int j = 0; j < kThreads / 32; ++j) {
    const bool in = keys[j * 32 + lane] >= bound;
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (in) sh.sel[at + __popc(m & ((1u << lane) - 1u))] = j * 32 + lane;
    at += __popc(m);
  }
  if (lane == 0) sh.nsel = at;
}

__device__ void select_columns(Shared& sh, int n, int lane) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < kThreads / 32; ++j) top = max(top, sh.vals[j * 32 + lane]);
  // 32 of the maxima, one a lane, reach the least of the lanes' largest
  const uint32_t lo = max(1u, __reduce_min_sync(0xffffffffu, top)), hi = max(lo, __reduce_max_sync(0xffffffffu, top));
  uint32_t bound;
  const bool ok = bisect<uint32_t>(sh.vals, n, lane, lo, hi, &bound);
  if (ok) list_columns<uint32_t>(sh, sh.vals, bound, lane);
  if (lane == 0) {
    sh.thr = (unsigned long long)bound << 32;
    sh.ties = !ok;
    sh.ncand = 0;
    sh.nunit = 0;
  }
}

// The entries of this CTA's slice [v0, v1) (vectors) that may be among its n
// largest, in sh.cand (sh.ncand of them; more than kCand where the list is full).
template <int DT>
__device__ void slice_candidates(Shared& sh, const char* row, int v0, int v1, int segs, int seg_slots, float mv, int mi, int n) {
  constexpr int N = Vec16<DT>::N;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (sh.ties) {  // full keys: the first entry equal to the maximum, in the slot where it appeared
    unsigned long long key = 0;
    for (int j = kUnroll - 1; j >= 0; --j) {
      const int i = mi + j * kThreads;
      if (v0 + tid < v1 && i < v1) {
        float v[N];
        Vec16<DT>::load(row + (size_t)i * 16, v);
#pragma unroll
        for (int e = N - 1; e >= 0; --e)
          if (v[e] == mv) key = entry_key(v[e], i * N + e);
      }
    }
    sh.keys[tid] = key;
    readers_sync();
    if (warp == 0) {
      const unsigned long long bound_value = sh.thr;
      unsigned long long bound;
      bisect<unsigned long long>(sh.keys, n, lane, bound_value, ~0ull, &bound);
      list_columns<unsigned long long>(sh, sh.keys, bound, lane);
      if (lane == 0) sh.thr = bound;
    }
    readers_sync();
  }
  const unsigned long long thr = sh.thr;
  const float floor = key_value(thr);
  for (int u = tid; u < sh.nsel * segs; u += kThreads) {
    const int col = sh.sel[u / segs], seg = u % segs;
    if (!(sh.seg_max[seg][col] < floor)) {
      const int c = atomicAdd(&sh.nunit, 1);
      if (c < kUnits) sh.units[c] = seg * kThreads + col;
    }
  }
  readers_sync();
  // vectors of a unit: every kThreads-th of its segment
  const bool listed = sh.nunit <= kUnits;
  const int per = listed ? seg_slots * kUnroll : (v1 - v0 + kThreads - 1) / kThreads;
  const int total = (listed ? sh.nunit : sh.nsel) * per;
  for (int q0 = tid; q0 < total; q0 += 4 * kThreads) {
    uint4 w[4];
    int at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int q = q0 + j * kThreads;
      at[j] = v1;
      if (q < total) {
        const int u = listed ? sh.units[q / per] : sh.sel[q / per];
        at[j] = v0 + u % kThreads + (u / kThreads * seg_slots * kUnroll + q % per) * kThreads;
      }
      if (at[j] < v1) w[j] = *reinterpret_cast<const uint4*>(row + (size_t)at[j] * 16);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (at[j] >= v1) continue;
      float v[N];
      Vec16<DT>::load(&w[j], v);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (!(v[e] < floor)) {  // a bound below every value decodes to NaN
          const unsigned long long k = entry_key(v[e], at[j] * N + e);
          if (k >= thr) {
            const int c = atomicAdd(&sh.ncand, 1);
            if (c < kCand) sh.cand[c] = k;
          }
        }
      }
    }
  }
  readers_sync();
}

// Calls put(rank, key) for the n largest keys of the slice.
template <int DT, typename Put>
__device__ __forceinline__ void slice_top(Shared& sh, const char* row, int v0, int v1, int n, Put put) {
  constexpr int N = Vec16<DT>::N;
  const int tid = threadIdx.x;
  const int cnt = sh.ncand;
  if (cnt <= kCand) {
    for (int c = tid; c < cnt; c += kThreads) {
      const unsigned long long k = sh.cand[c];
      int r = 0;
      for (int j = 0; j < cnt && r < n; ++j) r += sh.cand[j] > k;
      if (r < n) put(r, k);
    }
  } else {  // very many entries above the bound: one at a time, largest first
    const int per = (v1 - v0 + kThreads - 1) / kThreads;
    unsigned long long last = ~0ull;
    for (int r = 0; r < n; ++r) {
      unsigned long long best = 0;
      for (int q = tid; q < sh.nsel * per; q += kThreads) {
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
      if (!last) break;
      if (tid == 0) put(r, last);
    }
  }
}

// s and t of a whole row whose maximum m is known, entry by entry in the plain
// form (rows whose maximum's z would be rounded too far; b256 j5 v129280 at
// temperature 1e-6 125 us, 62 at 1).
template <int DT>
__device__ void plain_sums(Shared& sh, const char* row, int nvec, float cs, RowStat& c) {
  constexpr int N = Vec16<DT>::N;
  float s = 0.f, t = 0.f;
  for (int i = threadIdx.x; i < nvec; i += kThreads) {
    float v[N];
    Vec16<DT>::load(row + (size_t)i * 16, v);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float z = v[e] == -INFINITY ? kFloorZ : zdiff(v[e], c.m, cs);
      const float w = ex2(z);
      s += w;
      t = fmaf(w, z, t);
    }
  }
  s = warp_sum(s);
  t = warp_sum(t);
  readers_sync();
  if ((threadIdx.x & 31) == 0) sh.warp_stat[threadIdx.x >> 5] = {c.m, s, t, c.chk};
  readers_sync();
  c.s = c.t = 0.f;
  for (int w = 0; w < kThreads / 32; ++w) {
    c.s += sh.warp_stat[w].s;
    c.t += sh.warp_stat[w].t;
  }
}

// A cluster of C CTAs takes a row; CTA q reads vectors [q per, (q + 1) per).
template <int DT>
__global__ void __launch_bounds__(kThreads + 32, kCtasPerSm) logprobs_kernel(LogprobArgs a, int C) {
  extern __shared__ __align__(128) unsigned char shared_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(shared_raw);
  constexpr int N = Vec16<DT>::N;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_wait();
  const long long r = blockIdx.x / C;
  const int q = blockIdx.x % C;
  const int b = (int)(r / a.J);
  const int tok = a.tok[r], n = a.n_top;
  const float tau = a.temp ? a.temp[b] : 1.f;
  const bool bad_tok = tok < -1 || tok >= a.V, bad_temp = !(tau >= 0.f && tau <= kMaxTemp);
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

  // The slice comes in slots of 16 KB, copied by the bulk-copy engine while the
  // readers work on the slots before. The feeding warp prepares the barriers and
  // starts at once.
  const int chunks = (max(0, v1 - v0) + kSlotVecs - 1) / kSlotVecs;
  if (warp == kThreads / 32) {
    bool ok = true;
    int issued = 0;
    auto issue = [&](int c) {
      const int slot = c % kSlots, first = v0 + c * kSlotVecs, bytes = min(kSlotVecs, v1 - first) * 16;
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(&sh.full[slot])), "r"(bytes) : "memory");
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(saddr(sh.ring[slot])),
          "l"(row + (size_t)first * 16), "r"(bytes), "r"(saddr(&sh.full[slot]))
          : "memory");
      ++issued;
    };
    if (lane == 0) {
      for (int i = 0; i < kSlots; ++i) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(saddr(&sh.full[i])) : "memory");
        asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(&sh.empty[i])), "r"(kThreads / 32) : "memory");
      }
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      sh.dead = 0;
      for (int c = 0; c < min(chunks, kSlots); ++c) issue(c);
    }
    __syncthreads();
    if (lane == 0) {
      for (int c = kSlots; c < chunks; ++c) {
        ok = mbar_wait_bounded(saddr(&sh.empty[c % kSlots]), (c / kSlots - 1) & 1);
        if (!ok) break;
        issue(c);
      }
      if (!ok) {
        report_wait(a.status, kWhereEmpty, b);
        *(volatile int*)&sh.dead = 1;
        for (int c = max(0, issued - kSlots); c < issued; ++c)  // let issued copies land before the CTA exits
          mbar_wait_bounded(saddr(&sh.full[c % kSlots]), (c / kSlots) & 1);
      }
    }
    __syncwarp();
  } else {
    __syncthreads();
  }

  using W = Words<DT>;
  constexpr int kPairs = N / 2;
  RowStat st = {-INFINITY, 0.f, 0.f, -INFINITY};
  const float reach = kClampZ / cs;
  const f32x2 cs2 = pack2(cs, cs);
  float mz = 0.f;                                        // the maximum's z, rounded
  bool scaled = false;                                   // the sums are those of mz (else nothing is in them)
  f32x2 neg_mz = 0, s2[2] = {0, 0}, t2[2] = {0, 0};      // sums of 2^z', z' 2^z' with z' = l cs - mz, both halves
  uint32_t low = W::floor_of(-reach);
  int mi = v0 + tid;

  const int seg_slots = max(1, (chunks + kSegs - 1) / kSegs), segs = (chunks + seg_slots - 1) / seg_slots;
  float seg_m = -INFINITY;  // of the current segment, with seg_left slots to come
  int seg = 0, seg_left = seg_slots;

  auto batch = [&](uint32_t (&v)[kUnroll][4], int i, bool last) {
    uint32_t b2[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b2[e] = W::max_nan(W::max_nan(v[0][e], v[1][e]), W::max_nan(v[2][e], v[3][e]));
    const float bm = W::top(W::max_nan(W::max_nan(b2[0], b2[1]), W::max_nan(b2[2], b2[3])));
    st.chk = max_nan(st.chk, bm);
    if (n) {
      seg_m = fmaxf(seg_m, bm);
      if (--seg_left == 0 || last) {
        sh.seg_max[seg++][tid] = seg_m;
        seg_m = -INFINITY;
        seg_left = seg_slots;
      }
    }
    if (bm > st.m) {
      // a maximum whose z is too large to round adds nothing here: another column's is
      // larger by 2^22 or more, or the row takes the plain pass
      const bool fits = fabsf(bm) * cs < kFarZ;
      const float bz = fits ? bm * cs : 0.f, d = fmaxf(scaled ? mz - bz : kFloorZ, kFloorZ), f = ex2(d);
      const f32x2 d2 = pack2(d, d), f2 = pack2(f, f);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        t2[e] = mul2(f2, fma2(d2, s2[e], t2[e]));
        s2[e] = mul2(f2, s2[e]);
      }
      st.m = bm;
      mi = i;
      mz = bz;
      scaled = fits;
      neg_mz = pack2(-bz, -bz);
      low = W::floor_of(fits ? __fsub_rd(bm, reach) : -reach);
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j][e] = W::max_num(v[j][e], low);
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        const f32x2 z2 = fma2(W::pair(v[j], e), cs2, neg_mz);
        float za, zb;
        unpack2(z2, za, zb);
        const f32x2 w2 = pack2(ex2(za), ex2(zb));
        s2[e & 1] = add2(s2[e & 1], w2);
        t2[e & 1] = fma2(w2, z2, t2[e & 1]);
      }
    }
  };

  if (warp < kThreads / 32) {
    int slot = 0, i = v0 + tid;
    uint32_t ph = 0;
    for (int c = 0; c < chunks; ++c, i += kSlotVecs) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(saddr(&sh.full[slot]), ph))) {
        if (lane == 0 && !*(volatile int*)&sh.dead) report_wait(a.status, kWhereFull, b);
        *(volatile int*)&sh.dead = 1;
        break;
      }
      uint32_t v[kUnroll][4];
      const uint4* src = &sh.ring[slot][tid];
      auto take = [&](int j) {
        const uint4 x = src[j * kThreads];
        v[j][0] = x.x;
        v[j][1] = x.y;
        v[j][2] = x.z;
        v[j][3] = x.w;
      };
      if (c + 1 < chunks) {
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) take(j);
      } else {
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
          v[j][0] = v[j][1] = v[j][2] = v[j][3] = W::kNegInf;
          if (i + j * kThreads < v1) take(j);
        }
      }
      __syncwarp();
      if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(&sh.empty[slot])) : "memory");
      batch(v, i, c + 1 == chunks);
      if (++slot == kSlots) {
        slot = 0;
        ph ^= 1;
      }
    }
    float a0, a1, b0, b1;
    unpack2(add2(s2[0], s2[1]), a0, a1);
    unpack2(add2(t2[0], t2[1]), b0, b1);
    // z' = z + e with e = m cs - mz, the rounding of mz
    const float e = scaled ? fmaf(st.m, cs, -mz) : 0.f, f = ex2(-e);
    st.s = f * (a0 + a1);
    st.t = f * ((b0 + b1) - e * (a0 + a1));
  }

  cg::cluster_group cluster = cg::this_cluster();
  if (C > 1) cluster.sync();  // CTA 0's shared memory exists before it is written
  Shared* root = C > 1 ? cluster.map_shared_rank(&sh, 0) : &sh;
  const bool reader = warp < kThreads / 32;
  const int mv_i = mi;
  const float mv = st.m;
  if (reader) {
    if (n) sh.vals[tid] = v0 + tid < v1 ? value_key(mv) : 0;
    if (n && tid < n) root->lists[q * n + tid] = 0;
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
    readers_sync();
    if (warp == 0 && n) select_columns(sh, n, lane);
    if (warp == 1 && lane == 0) {
      RowStat c = sh.warp_stat[0];
      for (int w = 1; w < kThreads / 32; ++w) c = stat_merge(c, sh.warp_stat[w], cs);
      root->cta_stat[q] = c;
    }
    readers_sync();
    if (n) slice_candidates<DT>(sh, row, v0, v1, segs, seg_slots, mv, mv_i, n);
    if (n && C > 1) slice_top<DT>(sh, row, v0, v1, n, [&](int rank, unsigned long long k) { root->lists[q * n + rank] = k; });
  }
  if (C > 1) cluster.sync();
  if (q != 0 || !reader) return;

  RowStat c = sh.cta_stat[0];
  for (int w = 1; w < C; ++w) c = stat_merge(c, sh.cta_stat[w], cs);
  const bool bad = c.chk != c.chk || c.m == INFINITY || c.m == -INFINITY || sh.dead;
  if (!bad && !(fabsf(c.m) * cs < kPlainZ)) plain_sums<DT>(sh, row, nvec, cs, c);
  const float ln_s = logf(c.s);
  if (tid == 0) {
    if (bad && !sh.dead) report(a.status, DSPARK_STATUS_BAD_ROW, b);
    const float l = Elem<DT>::load(reinterpret_cast<const typename Elem<DT>::T*>(row), tok);
    a.logp[r] = bad ? 0.f : (l - c.m) / temp - ln_s;
    if (a.entropy) a.entropy[r] = bad ? 0.f : fmaxf(0.f, ln_s - kLn2 * (c.t / c.s));
    if (a.lse) a.lse[r] = bad ? 0.f : c.m / temp + ln_s;
  }
  if (bad) {
    if (tid < n) {
      a.top_idx[r * n + tid] = -1;
      a.top_logp[r * n + tid] = -INFINITY;
    }
    return;
  }
  auto put = [&](int rank, unsigned long long key) {
    a.top_idx[r * n + rank] = key_index(key);
    a.top_logp[r * n + rank] = (key_value(key) - c.m) / temp - ln_s;
  };
  if (C == 1) {
    if (n) slice_top<DT>(sh, row, v0, v1, n, put);
  } else {
    for (int k = tid; k < C * n; k += kThreads) {
      const unsigned long long key = sh.lists[k];
      int rank = 0;
      for (int j = 0; j < C * n; ++j) rank += sh.lists[j] > key;
      if (key && rank < n) put(rank, key);
    }
  }
}

// dlogits = (1 / temp) [ g_logp (1[v = tok] - p) - g_entropy p (ln p + H) ] with
// ln p = l / temp - lse: elementwise, so a read and a write of the logits. The
// sums of the forward pass come back as lse and H. An entry is p (c0 + c1 ln p)
// with c1 = -g_entropy / temp, c0 = -g_logp / temp + c1 H, on packed pairs; the
// token's entry alone gets g_logp / temp on top. A CTA takes one part of a row, so
// that the row's scalars are read once for many vectors, and loads a batch of
// vectors while it works on the one before.
constexpr int kGradVecs = 4;                              // vectors of a thread in a batch
constexpr int kGradBatch = kThreads * kGradVecs;
constexpr int kGradBatches = 2;                           // batches of a part, at most (8: 109 us, 2: 102 us at b256 j5 v129280)

// lse carries p = exp(l / temp - lse) with an error of 2^-24 |lse|, and 1 / temp one of
// the same size: 2^-11 at this bound, a quarter of a bf16 rounding. Past it (temperatures
// below about 0.01, logits far from zero) one CTA takes the row, so that dlogits may still
// be logits, and forms the maximum and the sum again (b256 j5 v129280 504 us, 99 below the
// bound; b1 j5 126 us and 10.5).
constexpr float kFarLse = 4096.f;
constexpr float kFarInv = 1.0e30f;  // 1 / temp past this would overflow in the products

template <int DT>
__device__ __noinline__ void grad_far_row(const char* row, char* out, int nvec, Status* status, int b, int tok, float temp, float gl,
                                          float gh, float H) {
  constexpr int N = Vec16<DT>::N;
  __shared__ float red[2][kThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float m = -INFINITY, s = 0.f;
  for (int i = tid; i < nvec; i += kThreads) {
    float v[N];
    Vec16<DT>::load(row + (size_t)i * 16, v);
#pragma unroll
    for (int e = 0; e < N; ++e) m = max_nan(m, v[e]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
  for (int w = 0; w < kThreads / 32; ++w) m = max_nan(m, red[0][w]);
  const bool bad = !(fabsf(m) < INFINITY);  // not the logits that lse was made of
  if (bad && tid == 0) report(status, DSPARK_STATUS_BAD_ROW, b);
  const float cs = fminf(kLog2e / temp, 3.0e38f);
  for (int i = tid; i < nvec; i += kThreads) {
    float v[N];
    Vec16<DT>::load(row + (size_t)i * 16, v);
#pragma unroll
    for (int e = 0; e < N; ++e) s += ex2(zdiff(v[e], m, cs));
  }
  s = warp_sum(s);
  if (lane == 0) red[1][warp] = s;
  __syncthreads();  // every entry has been read twice: the output may take the logits' place
  s = 0.f;
  for (int w = 0; w < kThreads / 32; ++w) s += red[1][w];
  const float ln_s = logf(s);
  for (int i = tid; i < nvec; i += kThreads) {
    float v[N];
    Vec16<DT>::load(row + (size_t)i * 16, v);
    alignas(16) typename Elem<DT>::T o[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float lp = fmaxf((v[e] - m) / temp, -200.f) - ln_s, p = ex2(lp * kLog2e);
      const float d = ((i * N + e == tok ? gl : 0.f) - p * fmaf(gh, lp + H, gl)) / temp;
      o[e] = Elem<DT>::store_round(bad ? 0.f : d);
    }
    *reinterpret_cast<uint4*>(out + (size_t)i * 16) = *reinterpret_cast<const uint4*>(o);
  }
}

template <int DT, bool ENTROPY>
__global__ void __launch_bounds__(kThreads, 5) logprobs_grad_kernel(LogprobGradArgs a, int parts, int batches) {
  constexpr int N = Vec16<DT>::N, kPairs = N / 2;
  using W = Words<DT>;
  grid_wait();
  const int nvec = a.V / N;
  const long long r = blockIdx.x / parts;
  const int part = blockIdx.x % parts, b = (int)(r / a.J);
  const int tok = a.tok[r];
  const float tau = a.temp ? a.temp[b] : 1.f;
  const float lse = a.lse[r], gl = a.g_logp[r];
  const float gh = ENTROPY ? a.g_entropy[r] : 0.f, H = ENTROPY ? a.entropy[r] : 0.f;
  const bool bad_tok = tok < -1 || tok >= a.V, bad_temp = !(tau >= 0.f && tau <= kMaxTemp);
  const bool bad_row = !(fabsf(lse) < INFINITY);
  const char* row = static_cast<const char*>(a.logits) + r * a.V * Elem<DT>::kBytes;
  char* out = static_cast<char*>(a.dlogits) + r * a.V * Elem<DT>::kBytes;
  const int i0 = part * batches * kGradBatch + threadIdx.x, i1 = min(nvec, (part + 1) * batches * kGradBatch);
  if (tok < 0 || bad_tok || bad_temp || bad_row) {
    if (tok != -1 && part == 0 && threadIdx.x == 0)
      report(a.status, bad_tok ? DSPARK_STATUS_BAD_TOKEN : bad_temp ? DSPARK_STATUS_BAD_TEMP : DSPARK_STATUS_BAD_ROW, b);
    for (int i = i0; i < i1; i += kThreads) *reinterpret_cast<uint4*>(out + (size_t)i * 16) = make_uint4(0, 0, 0, 0);
    return;
  }
  const float temp = tau > 0.f ? tau : 1.f, inv = 1.f / temp;
  if (!(fabsf(lse) < kFarLse && inv < kFarInv)) {
    if (part == 0) grad_far_row<DT>(row, out, nvec, a.status, b, tok, temp, gl, gh, H);
    return;
  }
  const float c1 = -gh * inv, c0 = fmaf(c1, H, -gl * inv);
  const f32x2 inv2 = pack2(inv, inv), lse2 = pack2(-lse, -lse), e2 = pack2(kLog2e, kLog2e);
  const f32x2 c02 = pack2(c0, c0), c12 = pack2(c1, c1);
  const int tok_vec = tok / N;

  uint4 next[kGradVecs];
  auto load = [&](int i) {
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j)
      if (i + j * kThreads < i1) next[j] = __ldcs(reinterpret_cast<const uint4*>(row) + i + j * kThreads);
  };
  load(i0);
  for (int i = i0; i < i1; i += kGradBatch) {
    uint4 x[kGradVecs];
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) x[j] = next[j];
    load(i + kGradBatch);
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
      const int iv = i + j * kThreads;
      if (iv >= i1) continue;
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      float d[N];
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        f32x2 lp = fma2(W::pair(w, e), inv2, lse2);
        float la, lb;
        if (ENTROPY) {  // -inf is p = 0 here, not 0 * inf; exp(-200) is zero in fp32
          unpack2(lp, la, lb);
          lp = pack2(fmaxf(la, -200.f), fmaxf(lb, -200.f));
        }
        unpack2(mul2(lp, e2), la, lb);
        const f32x2 p = pack2(ex2(la), ex2(lb));
        unpack2(mul2(p, ENTROPY ? fma2(c12, lp, c02) : c02), d[2 * e], d[2 * e + 1]);
      }
      if (iv == tok_vec) {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (iv * N + e == tok) d[e] = fmaf(gl, inv, d[e]);
      }
      alignas(16) typename Elem<DT>::T o[N];
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = Elem<DT>::store_round(d[e]);
      *reinterpret_cast<uint4*>(out + (size_t)iv * 16) = *reinterpret_cast<const uint4*>(o);
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
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
  if (e != cudaSuccess) return e;
  return launch_early(kern, dim3((unsigned)(rows * C)), kThreads + 32, (int)sizeof(Shared), C, s, a, C);
}

cudaError_t logprobs_grad_launch(const LogprobGradArgs& a, int num_sms, cudaStream_t s) {
  const long long rows = (long long)a.B * a.J;
  const int nvec = a.V / (a.dtype == DSPARK_F32 ? 4 : 8);
  // parts of up to kGradBatches batches, fewer while that leaves SMs without one
  int batches = min(kGradBatches, (nvec + kGradBatch - 1) / kGradBatch);
  auto parts_of = [&](int n) { return (nvec + n * kGradBatch - 1) / (n * kGradBatch); };
  while (batches > 1 && rows * parts_of(batches) < 4LL * num_sms) batches /= 2;
  const int parts = parts_of(batches);
  const bool f32 = a.dtype == DSPARK_F32, ent = a.g_entropy != nullptr;
  auto kern = f32 ? (ent ? logprobs_grad_kernel<DSPARK_F32, true> : logprobs_grad_kernel<DSPARK_F32, false>)
                  : (ent ? logprobs_grad_kernel<DSPARK_BF16, true> : logprobs_grad_kernel<DSPARK_BF16, false>);
  if (rows * parts > INT_MAX) return cudaErrorInvalidValue;
  return launch_early(kern, dim3((unsigned)(rows * parts)), kThreads, 0, 1, s, a, parts, batches);
}

}  // namespace dspark
