// Linear product with scales, bias, activation and residual in its epilogue, and
// its gradient, on the tensor cores (tcgen05, operands by TMA).
//
//   y[m, n] = act(x_scale[m] w_scale[n] sum_k x[m, k] w[n, k] + bias[n]) + residual[m, n]
//   dpre = dy act'(pre), dx = dpre w, dw = dpre^T x, dbias = column sums of dpre
//
// Orientation: the matrix instruction's 128 rows (tensor-memory lanes) are the
// output's contiguous index (features), its columns the other one (tokens).
// One kernel then serves one token and thousands: the column tile is 16 to 256
// wide, and a small batch streams the weights past a few columns. The three products differ
// only in which operand lies contraction-major:
//   y  [m, n]: lanes n, A = w (k contiguous),  columns m, B = x    (k contiguous)
//   dx [m, k]: lanes k, A = w (k = lanes contiguous), columns m, B = dpre (n contiguous)
//   dw [n, k]: lanes k, A = x (k = lanes contiguous), columns n, B = dpre (n = columns contiguous)
//
// Persistent pairs of CTAs (cta_group::2: one matrix instruction of 256 lanes
// uses both SMs' tensor cores, each SM holding its 128 lanes of A and of the
// result and half of B's columns, so every B byte enters one SM only) take work
// units (an output tile or part of its contraction):
//   warp 0     TMA producer: 128-byte-wide boxes of this CTA's A and B into a ring
//              of stages; the bytes of both CTAs complete on the first one's barrier
//   warp 1     tensor-memory allocation and, in the first CTA, the single-thread
//              tcgen05.mma issuer
//   warps 2-9  epilogue of the previous unit meanwhile (two accumulators): a warp
//              reads its quarter of the lanes (hardware: warp index mod 4), the two
//              warps of a quarter take blocks of 32 columns in turn
// With few tiles a cluster of 2, 4 or 8 pairs takes one tile, each pair a part of
// the contraction; the other pairs leave their fp32 sums in the first one's shared
// memory (its ring is free by then), which adds them in the order of the parts and
// finishes the tile.
// Measured in steady repeats, under the power cap (in brackets: ten calls from a cool
// chip): m1536 n129280 k4096 1222 us in bf16 (1063; 1.33 PFLOP/s), 667 us in e4m3 (581;
// 2.44 PFLOP/s); m16 n129280 k4096 164 us (6.5 TB/s, memory bounds it); gradient
// m2048 n5120 k4096 with gelu 159 us (137). The other figures of this file come from
// short runs of both sides in turn.
// Every wait is bounded; a CTA that gives up reports DSPARK_STATUS_TIMEOUT.
#include "host.cuh"
#include "launch.cuh"
#include "linear.cuh"
#include "norm.cuh"
#include "tcgen05.cuh"

namespace dspark {

namespace {

using namespace t5;

constexpr int kEpiWarps = 8;                   // two per quarter of the lanes (more would halve the registers of a thread)
constexpr int kEpiThreads = 32 * kEpiWarps;
constexpr int kThreads = 64 + kEpiThreads;
constexpr int kTileF = 256;                    // lanes: output features per tile, 128 in each CTA of the pair
constexpr int kLanes = 128;
constexpr int kMaxCols = 256;                  // columns per tile at most
constexpr int kABytes = kLanes * 128;          // A of a stage: 128 bytes of contraction (or lanes) x 128
constexpr int kMaxStages = 12;
constexpr int kRing = 6 * 32768;               // bytes of the stage ring
constexpr int kBoxBytes = 64 * 128;            // one [64 x 128 bytes] box of a lane- or column-contiguous operand
constexpr int kChunk = 32;                     // columns that an epilogue warp takes at a time
constexpr int kStageBytes = kChunk * 64;       // a warp's staged chunk: 32 columns x 32 lanes of 2 bytes
constexpr int kOffStage = kRing;
constexpr int kOffBar = kOffStage + kEpiWarps * kStageBytes;
constexpr int kNumBars = 2 * kMaxStages + 4;
constexpr int kSmem = kOffBar + kNumBars * 8 + 16;
static_assert(kSmem <= 232448, "exceeds the 227 KB of shared memory per block");
constexpr int kPlanPairs = 74;                 // pairs of SMs that the split of the work is planned for

enum : unsigned int {  // wait sites recorded when a bounded wait gives up
  kWhereEmpty = 40,
  kWhereFull = 41,
  kWhereAccFull = 42,
  kWhereAccEmpty = 43,
};

struct Gemm {
  int F, T;                 // lanes (contiguous outputs) and columns in all
  int kblocks;              // 128-byte (K-major) or 64-row (otherwise) blocks of the contraction
  int nt;                   // columns per tile, a multiple of 16 (32 when B is column-contiguous)
  int tiles_f, tiles_t;
  int parts;                // pairs that share a tile (1, 2, 4 or 8)
  const float* col_scale;   // [T] or null
  const float* lane_scale;  // [F] or null
  const float* bias;        // [F] or null
  const void* residual;     // [T, F] or null
  void* out;                // [T, F]
  void* pre;                // [T, F] or null
  int out_type, act;
  Order order;
  Status* status;
};

// z / (1 + exp(-v)) by a power of two and the fast division (together 2^-21 of the result
// and 2^-23 |v|; also where the output is fp32): silu with v = z, gelu's tanh form with v = 2 sqrt(2/pi) (z + 0.044715 z^3)
__device__ __forceinline__ float gate(float z, float v) { return __fdividef(z, 1.f + ex2(-v * kLog2e)); }

constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// act'(z). At |z| = 128 the gates are 0 or 1 exactly (2^184 is infinite in fp32), and
// so they stay for larger |z|, whose cubes and products would overflow
__device__ __forceinline__ float activate_grad(float z, int act) {
  if (act == DSPARK_ACT_RELU) return z > 0.f ? 1.f : (z != z ? z : 0.f);
  z = z != z ? z : fminf(fmaxf(z, -128.f), 128.f);
  const float v = act == DSPARK_ACT_SILU ? z : kGelu2 * fmaf(0.044715f * z * z, z, z);
  const float dv = act == DSPARK_ACT_SILU ? 1.f : kGelu2 * fmaf(3.f * 0.044715f * z, z, 1.f);
  const float g = __fdividef(1.f, 1.f + ex2(-v * kLog2e));
  return g + z * g * (1.f - g) * dv;
}

template <int N>
__device__ __forceinline__ void activate(float* v, int act) {
  if (act == DSPARK_ACT_RELU) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = v[j] < 0.f ? 0.f : v[j];  // NaN stays
  } else if (act == DSPARK_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = gate(v[j], v[j]);
  } else if (act == DSPARK_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = gate(v[j], kGelu2 * fmaf(0.044715f * v[j] * v[j], v[j], v[j]));
  }
}

// fp32 outputs (and 2-byte rows that are not whole 16-byte vectors): 16 columns
// of one lane straight to memory, 32 neighbouring outputs per warp and store. at:
// column 0; n columns. Residuals come as bits, loaded a chunk ahead: a load behind
// a store that might alias it would wait for its turn.
template <int DT>
__device__ __forceinline__ void direct_load16(const Gemm& g, uint32_t* res, long long at, int n) {
  using T = typename Elem<DT>::T;
  const T* p = static_cast<const T*>(g.residual) + at;
#pragma unroll
  for (int j = 0; j < 16; ++j, p += g.F)
    if (j < n) res[j] = DT == DSPARK_F32 ? __float_as_uint((float)*p) : (uint32_t)*p;
}
template <int DT>
__device__ __forceinline__ void direct16(const Gemm& g, float* v, const uint32_t* res, long long at, int n) {
  using T = typename Elem<DT>::T;
  if (g.pre) {
    T* p = static_cast<T*>(g.pre) + at;
#pragma unroll
    for (int j = 0; j < 16; ++j, p += g.F)
      if (j < n) *p = Elem<DT>::store_round(v[j]);
  }
  activate<16>(v, g.act);
  if (g.residual) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < n) v[j] += __uint_as_float(DT == DSPARK_F32 ? res[j] : res[j] << 16);
  }
  T* p = static_cast<T*>(g.out) + at;
#pragma unroll
  for (int j = 0; j < 16; ++j, p += g.F)
    if (j < n) *p = Elem<DT>::store_round(v[j]);
}

// bf16 outputs whose rows are whole 16-byte vectors go through shared memory: a
// lane holds features of many tokens, memory wants many features of one token.
// A warp's stage is its own (no barrier but the warp's): row r is token t0 + r,
// 32 features in four 16-byte vectors, vector q at q ^ (r / 2 % 4), so that eight
// rows of one vector and two rows of four both fall on all banks.
__device__ __forceinline__ uint32_t stage_at(int r, int q) { return r * 64 + ((q ^ ((r >> 1) & 3)) << 4); }

// Moves rows between a warp's stage and memory (p: token t0, the warp's first
// feature; nf features of the row remain): 8 rows x 64 bytes an instruction. Loads
// go through registers, so that they can be started long before.
__device__ __forceinline__ void load_rows(uint4* x, const uint16_t* p, int F, int nf, int rows, int lane) {
  const int q = lane & 3;
  if (q * 8 >= nf) return;
  p += (long long)(lane >> 2) * F + q * 8;
#pragma unroll
  for (int i = 0; i < kChunk / 8; ++i)
    if (i * 8 + (lane >> 2) < rows) x[i] = *reinterpret_cast<const uint4*>(p + (long long)(i * 8) * F);
}
__device__ __forceinline__ void stage_rows(unsigned char* stage, const uint4* x, int lane) {
#pragma unroll
  for (int i = 0; i < kChunk / 8; ++i)
    *reinterpret_cast<uint4*>(stage + stage_at(i * 8 + (lane >> 2), lane & 3)) = x[i];
}
__device__ __forceinline__ void store_rows(const unsigned char* stage, uint16_t* p, int F, int nf, int rows, int lane) {
  const int q = lane & 3;
  if (q * 8 >= nf) return;
  p += (long long)(lane >> 2) * F + q * 8;
#pragma unroll
  for (int i = 0; i < kChunk / 8; ++i) {
    const int r = i * 8 + (lane >> 2);
    if (r < rows) *reinterpret_cast<uint4*>(p + (long long)(i * 8) * F) = *reinterpret_cast<const uint4*>(stage + stage_at(r, q));
  }
}

// The tiles of a pair: `first`, `first + step`, ... . Tiles run over the columns
// first, so that pairs working at the same time share their rows of A. Steps by
// additions: a tile of a short contraction lasts less than two divisions.
struct Tiles {
  int tf, tt, left, dtt, dtf;
  __device__ __forceinline__ Tiles(const Gemm& g, int first, int step) {
    const int tiles = g.tiles_f * g.tiles_t;
    left = tiles > first ? (tiles - first + step - 1) / step : 0;
    tt = first % g.tiles_t;
    tf = first / g.tiles_t;
    dtt = step % g.tiles_t;
    dtf = step / g.tiles_t;
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next(const Gemm& g) {
    --left;
    tt += dtt;
    tf += dtf;
    if (tt >= g.tiles_t) {
      tt -= g.tiles_t;
      ++tf;
    }
  }
};

// A_MN / B_MN: the operand is contiguous along lanes / columns, not along the contraction.
// STAGED: bf16 rows of whole 16-byte vectors, through shared memory.
template <bool F8, bool A_MN, bool B_MN, bool STAGED>
__global__ void __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, Gemm g) {
  extern __shared__ __align__(1024) unsigned char smem[];
  if (su32(smem) & 1023u) {  // 128-byte-swizzled tiles need 1024-byte alignment (the same offset in every CTA)
    grid_wait();
    if (threadIdx.x == 0) report(g.status, DSPARK_STATUS_INTERNAL, 0);
    return;
  }
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  volatile int* dead = abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t cluster_rank = cta_rank(), rank = cluster_rank & 1;  // rank: CTA of the pair
  const uint32_t first_rank = cluster_rank & ~1u;
  const uint16_t both = (uint16_t)(3u << first_rank);
  const int part = cluster_rank >> 1;  // the pair's part of the contraction
  const int kb0 = (int)((long long)g.kblocks * part / g.parts), kb1 = (int)((long long)g.kblocks * (part + 1) / g.parts);
  const int nh = g.nt / 2;  // columns of B in this CTA
  const int stage_bytes = kABytes + (B_MN ? (nh + 63) / 64 * kBoxBytes : nh * 128);
  const int stages = min(kMaxStages, kRing / stage_bytes);
  Tiles w(g, blockIdx.x / (2 * g.parts), gridDim.x / (2 * g.parts));

  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * kEpiThreads / 32);  // a warp of either CTA each
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {  // two accumulators of 256 columns
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  fence_before();
  cluster_sync();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  if (g.order == kAfter) grid_wait();
  grid_release();  // behind the wait: a launch beside this one relies on the same results

  // The producer's and the issuer's loop have to keep up with a block of 512
  // tensor-core cycles: they run in a whole converged warp, of which one lane
  // issues, stages and phases are counted, not divided, and addresses and
  // descriptors advance by additions (a loop of one thread that computed them
  // anew took 730 cycles a block).
  if (warp == 0) {
    const bool lead = elect_one();
    const uint32_t smem0 = su32(smem), full0 = map_rank(su32(full), first_rank);
    int s = 0, issued = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (; w.more() && ok; w.next(g)) {
      const int f0 = w.tf * kTileF + rank * kLanes, t0 = w.tt * g.nt + rank * nh;
      int kx = kb0 * (F8 ? 128 : 64);
      for (int kb = kb0; kb < kb1; ++kb, kx += F8 ? 128 : 64) {
        ok = mbar_wait_warp(&empty[s], ph);
        if (!ok) break;
        if (lead) {
          if (rank == 0) mbar_expect_tx(&full[s], 2 * stage_bytes);
          const uint32_t bar = full0 + 8 * s;
          const uint32_t a = smem0 + s * stage_bytes, b = a + kABytes;
          if (A_MN) {
            tma_load_2d(a, &map_a, f0, kx, bar);
            tma_load_2d(a + kBoxBytes, &map_a, f0 + 64, kx, bar);
          } else {
            tma_load_2d(a, &map_a, kx, f0, bar);
          }
          if (B_MN) {
            for (int q = 0; q < (nh + 63) / 64; ++q) tma_load_2d(b + q * kBoxBytes, &map_b, t0 + q * 64, kx, bar);
          } else {
            tma_load_2d(b, &map_b, kx, t0, bar);
          }
        }
        __syncwarp();
        ++issued;
        if (++s == stages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok && lead) {
      if (!*dead) report_wait(g.status, kWhereEmpty, 0);
      *dead = 1;
      if (rank == 0)  // let issued loads of both CTAs land before the pair winds down (below)
        for (int q = max(0, issued - stages); q < issued; ++q) mbar_wait(&full[q % stages], (q / stages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      const bool lead = elect_one();
      // D fp32; A and B bf16 or e4m3; widths nt and 256
      const uint32_t idesc = (1u << 4) | (F8 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)A_MN << 15) |
                             ((uint32_t)B_MN << 16) | ((uint32_t)(g.nt >> 3) << 17) | ((uint32_t)(kTileF >> 4) << 24);
      // descriptors of the first stage; their low bits are the address in 16-byte units
      const uint64_t desc_a = A_MN ? sdesc(su32(smem), kBoxBytes, 1024) : sdesc(su32(smem), 16, 1024);
      const uint64_t desc_b = B_MN ? sdesc(su32(smem) + kABytes, kBoxBytes, 1024) : sdesc(su32(smem) + kABytes, 16, 1024);
      constexpr uint64_t step_a = (A_MN ? 2048 : 32) >> 4, step_b = (B_MN ? 2048 : 32) >> 4;
      int s = 0, done = 0;
      uint32_t ph = 0, aph = 1, buf = 0;
      uint64_t da = desc_a, db = desc_b;
      bool ok = true;
      unsigned int site = kWhereAccEmpty;
      for (; w.more(); w.next(g)) {
        ok = mbar_wait_warp(&acc_empty[buf], aph);
        if (!ok) break;
        fence_after();
        const uint32_t d = tmem + buf * kMaxCols;
        uint32_t acc = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = mbar_wait_warp(&full[s], ph);
          if (!ok) break;
          fence_after();
          if (lead) {
#pragma unroll
            for (int q = 0; q < 4; ++q)  // 32 bytes of the contraction (or 16 rows of it) each
              mma<F8>(d, da + q * step_a, db + q * step_b, idesc, q ? 1u : acc);
            mma_commit(&empty[s], both);
          }
          __syncwarp();
          acc = 1;
          ++done;
          da += stage_bytes >> 4;
          db += stage_bytes >> 4;
          if (++s == stages) {
            s = 0;
            ph ^= 1;
            da = desc_a;
            db = desc_b;
          }
        }
        if (!ok) {
          site = kWhereFull;
          break;
        }
        if (lead) mma_commit(&acc_full[buf], both);
        __syncwarp();
        buf ^= 1;
        if (buf == 0) aph ^= 1;
      }
      if (!ok && lead) {
        if (!*dead) report_wait(g.status, site, 0);
        *dead = 1;
        if (done > 0)  // MMAs complete in order: after the last commit tensor memory is quiet
          mbar_wait(&empty[(done - 1) % stages], ((done - 1) / stages) & 1);
      }
    }
    __syncwarp();
  }
  const uint32_t slots = (uint32_t)((g.nt + kChunk - 1) / kChunk * kChunk) * kLanes * 4;  // bytes of one part's sums
  if (g.parts > 1) {
    // one tile per cluster: when every pair's products are complete the rings are
    // free; sums of part q go to [q - 1, column, lane] of the first pair's
    const int quarter = warp & 3;
    const int c1 = min(g.nt, g.T - w.tt * g.nt);
    if (warp >= 2 && !mbar_wait(&acc_full[0], 0)) {
      if (!*dead) report_wait(g.status, kWhereAccFull, 0);
      *dead = 1;
    }
    __syncwarp();
    cluster_sync();
    if (warp >= 2 && part > 0) {
      fence_after();
      const uint32_t to = map_rank(su32(smem), rank) + (part - 1) * slots + (quarter * 32 + lane) * 4;
      for (int c = (warp - 2) / 4 * 16; c < c1; c += kEpiWarps / 4 * 16) {
        float v[16];
        tmem_ld_lanes(tmem + ((uint32_t)(quarter * 32) << 16) + c, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) st_cluster(to + (c + j) * kLanes * 4, v[j]);
      }
      fence_before();
    }
    cluster_sync();
  }
  if (warp >= 2 && part == 0) {
    const int quarter = warp & 3, group = (warp - 2) >> 2;
    const int ln = quarter * 32 + lane;    // lane of this CTA's part of the tile
    const uint32_t acc_free = map_rank(su32(acc_empty), first_rank);
    unsigned char* stage = smem + kOffStage + (warp - 2) * kStageBytes;
    const uint32_t mat = su32(stage) + stage_at(lane & 7, lane >> 3);  // + 512 for the next 8 columns
    // the features whose values this thread holds: one lane's, or four rows of its fragments
    constexpr int kRows = STAGED ? 4 : 1;
    constexpr int kCols = STAGED ? kChunk : 16;     // columns that a warp takes at a time
    constexpr int kStep = kEpiWarps / 4 * kCols;
    const int row0 = STAGED ? quarter * 32 + (lane >> 2) : ln;
    float ls[kRows], bias[kRows];

    // the residual of columns c .. c + kCols - 1, in the layout that finish() takes
    struct Residual {
      uint4 x[4];
    };
    auto load_residual = [&](Residual& res, int f0, int t0, int c) {
      const int cols = min(min(kCols, g.nt - c), g.T - t0 - c);
      if constexpr (STAGED) {
        const int fw = f0 + quarter * 32;
        load_rows(res.x, static_cast<const uint16_t*>(g.residual) + (long long)(t0 + c) * g.F + fw, g.F, g.F - fw, cols, lane);
      } else {
        const int n = f0 + ln < g.F ? cols : 0;
        const long long at = (long long)(t0 + c) * g.F + f0 + ln;
        uint32_t* bits = reinterpret_cast<uint32_t*>(res.x);
        if (g.out_type == DSPARK_F32)
          direct_load16<DSPARK_F32>(g, bits, at, n);
        else
          direct_load16<DSPARK_BF16>(g, bits, at, n);
      }
    };

    // columns c .. c + kCols - 1 of the tile to the outputs; cscale: lane j's is column j's scale
    auto finish = [&](float* v, const Residual& res, int f0, int t0, int c, float cscale) {
      const int cols = min(min(kCols, g.nt - c), g.T - t0 - c);
      if constexpr (!STAGED) {
        if (g.lane_scale) {
#pragma unroll
          for (int j = 0; j < kCols; ++j) v[j] *= ls[0] * __shfl_sync(0xffffffffu, cscale, j);
        }
        if (g.bias) {
#pragma unroll
          for (int j = 0; j < kCols; ++j) v[j] += bias[0];
        }
        const int n = f0 + ln < g.F ? cols : 0;
        const long long at = (long long)(t0 + c) * g.F + f0 + ln;
        if (g.out_type == DSPARK_F32)
          direct16<DSPARK_F32>(g, v, reinterpret_cast<const uint32_t*>(res.x), at, n);
        else
          direct16<DSPARK_BF16>(g, v, reinterpret_cast<const uint32_t*>(res.x), at, n);
      } else {
        if (g.lane_scale) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float s = __shfl_sync(0xffffffffu, cscale, 8 * k + 2 * (lane & 3) + e);
#pragma unroll
              for (int i = 0; i < 4; ++i) v[16 * (i >> 1) + 4 * k + 2 * (i & 1) + e] *= ls[i] * s;
            }
          }
        }
        if (g.bias) {
#pragma unroll
          for (int j = 0; j < kCols; ++j) v[j] += bias[2 * (j >> 4) + ((j >> 1) & 1)];
        }
        const int fw = f0 + quarter * 32;
        const long long at = (long long)(t0 + c) * g.F + fw;
        auto put = [&](void* p) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float* a = v + 16 * (i >> 1) + 4 * k + 2 * (i & 1);
              q[i] = pack_bf16x2(a[0], a[1]);
            }
            store_matrix_t(mat + k * 512, q);
          }
          __syncwarp();
          store_rows(stage, static_cast<uint16_t*>(p) + at, g.F, g.F - fw, cols, lane);
          __syncwarp();  // the stage is free again
        };
        if (g.pre) put(g.pre);
        activate<kCols>(v, g.act);
        if (g.residual) {
          stage_rows(stage, res.x, lane);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t q[4];
            load_matrix_t(mat + k * 512, q);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float* a = v + 16 * (i >> 1) + 4 * k + 2 * (i & 1);
              a[0] += __uint_as_float(q[i] << 16);
              a[1] += __uint_as_float(q[i] & 0xffff0000u);
            }
          }
          __syncwarp();
        }
        put(g.out);
      }
    };

    // A tile's residual (64 KB) is asked into L2 while the tile before is worked on:
    // a warp's own loads hold too few bytes to cover memory's latency.
    auto prefetch_residual = [&](const Tiles& at) {
      const int f0 = at.tf * kTileF + rank * kLanes, t = tid - 64, t0 = at.tt * g.nt;
      if (!at.more() || t >= g.nt || t0 + t >= g.T || f0 >= g.F) return;
      const int es = g.out_type == DSPARK_F32 ? 4 : 2, bytes = min(kLanes, g.F - f0) * es;
      const char* row = static_cast<const char*>(g.residual) + ((long long)(t0 + t) * g.F + f0) * es;
      for (int o = 0; o < bytes; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + o));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(row + bytes - 1));
    };
    if (g.residual) prefetch_residual(w);

    uint32_t buf = 0, aph = 0;
    for (; w.more(); w.next(g)) {
      if (g.residual) {
        Tiles after = w;
        after.next(g);
        prefetch_residual(after);
      }
      const int f0 = w.tf * kTileF + rank * kLanes, t0 = w.tt * g.nt;
      // scales and bias through L2 (__ldcg): the launch before, beside which this one may have
      // started, may have written them, and the read-only path's cache need not show that
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int f = f0 + row0 + 8 * i;
        ls[i] = g.lane_scale && f < g.F ? __ldcg(g.lane_scale + f) : 0.f;
        bias[i] = g.bias && f < g.F ? __ldcg(g.bias + f) : 0.f;
      }
      const int c1 = min(g.nt, g.T - t0);
      Residual next = {};
      if (g.residual && group * kCols < c1) load_residual(next, f0, t0, group * kCols);
      bool ok = !*dead;
      if (ok && !mbar_wait(&acc_full[buf], aph)) {
        ok = false;
        if (!*dead) report_wait(g.status, kWhereAccFull, 0);
        *dead = 1;
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      fence_after();
      const uint32_t src = tmem + buf * kMaxCols + ((uint32_t)(quarter * 32) << 16);
      for (int c = group * kCols; c < c1; c += kStep) {
        float v[kCols];
        const float cscale = g.col_scale && t0 + c + lane < g.T ? __ldcg(g.col_scale + t0 + c + lane) : 0.f;
        if constexpr (STAGED)
          tmem_ld_frags(src + c, v);
        else
          tmem_ld_lanes(src + c, v);
        if (c + kStep >= c1) {  // the warp's last chunk: its part of the accumulator is free
          fence_before();
          if (lane == 0) mbar_arrive_relaxed(acc_free + 8 * buf);
        }
        for (int q = 1; q < g.parts; ++q) {
          const float* s = reinterpret_cast<const float*>(smem + (q - 1) * slots) + c * kLanes;
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            if constexpr (STAGED)  // value j's column and lane in the fragments
              v[j] += s[(8 * (j >> 2 & 3) + 2 * (lane & 3) + (j & 1)) * kLanes + quarter * 32 + 16 * (j >> 4) + 8 * (j >> 1 & 1) + (lane >> 2)];
            else
              v[j] += s[j * kLanes + ln];
          }
        }
        const Residual res = next;
        if (g.residual && c + kStep < c1) load_residual(next, f0, t0, c + kStep);
        finish(v, res, f0, t0, c, cscale);
      }
      if (group * kCols >= c1 && lane == 0) mbar_arrive_relaxed(acc_free + 8 * buf);  // nothing to read
      buf ^= 1;
      if (buf == 0) aph ^= 1;
    }
  }
  fence_before();
  cluster_sync();  // neither CTA leaves while the other's arrivals or loads may still reach it
  fence_after();
  if (g.order == kBeside) grid_wait();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// dpre = round_bf16(dy act'(pre)) (the tensor cores take bf16 operands; the
// rounding is half a bf16 step of each factor, as in the bf16 result) and
// per-CTA column sums of the unrounded values. A CTA takes 256 columns and a
// contiguous run of rows, a warp every eighth row, four of them in flight.
constexpr int kDpreRows = 8, kDpreAhead = 4;

template <int ACT>
__global__ void __launch_bounds__(256) dpre_kernel(const void* dy, const void* pre, int M, int N, int rows_per, void* dpre,
                                                   float* partial) {
  __shared__ float part[kDpreRows][256 + 8];
  grid_release();
  grid_wait();
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int n0 = blockIdx.x * 256 + lane * 8;
  const int m1 = min(M, (int)(blockIdx.y + 1) * rows_per);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (n0 < N) {
    for (int m = blockIdx.y * rows_per + row; m < m1; m += kDpreRows * kDpreAhead) {
      uint4 d4[kDpreAhead], z4[kDpreAhead];
#pragma unroll
      for (int j = 0; j < kDpreAhead; ++j) {
        const size_t at = ((size_t)(m + j * kDpreRows) * N + n0) * 2;
        if (m + j * kDpreRows < m1) {
          d4[j] = *reinterpret_cast<const uint4*>(static_cast<const char*>(dy) + at);
          if (ACT != DSPARK_ACT_NONE) z4[j] = *reinterpret_cast<const uint4*>(static_cast<const char*>(pre) + at);
        }
      }
#pragma unroll
      for (int j = 0; j < kDpreAhead; ++j) {
        if (m + j * kDpreRows >= m1) continue;
        float d[8];
        Vec16<DSPARK_BF16>::load(&d4[j], d);
        if (ACT != DSPARK_ACT_NONE) {
          float z[8];
          Vec16<DSPARK_BF16>::load(&z4[j], z);
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] *= activate_grad(z[e], ACT);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(d[2 * e], d[2 * e + 1]);
          *reinterpret_cast<uint4*>(static_cast<char*>(dpre) + ((size_t)(m + j * kDpreRows) * N + n0) * 2) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += d[e];
      }
    }
  }
  if (!partial) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) part[row][lane * 8 + e] = acc[e];
  __syncthreads();
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n < N) {
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < kDpreRows; ++q) t += part[q][threadIdx.x];
    partial[(size_t)blockIdx.y * N + n] = t;
  }
}

// ---------------------------------------------------------------------------
// host: how the work is cut
// ---------------------------------------------------------------------------
struct Plan {
  int nt, tiles_f, tiles_t;
  int parts;     // pairs per tile
  int clusters;  // of 2 * parts CTAs
};

// The column width and the number of parts with the least time by measured costs
// in ns: a block of the contraction by its width (74 pairs, m1024 n18944, k2048
// against k1024; up to 64 columns the issuing loop bounds it); a tile at least its
// epilogue; the first loads and the last epilogue are not hidden; a joined tile has
// two cluster barriers and the parts' sums on top. The epilogue's cost is that of a plain
// staged one: a residual, pre, an activation or odd rows are not in it, and where the
// contraction is short they bound the tile (m1536 n64000 k512 with a residual takes 132 us
// where this says 79). Clusters of 2, 4, 8 and 16 CTAs
// of this size run 74, 33, 15 and 7 at once.
Plan make_plan(long long F, long long T, int kblocks, bool b_cols) {
  constexpr int kWidths[] = {16, 32, 48, 64, 96, 128, 160, 192, 224, 256};
  constexpr double kBlockNs[] = {150, 150, 150, 150, 193, 221, 253, 294, 354, 408};
  constexpr int kAtOnce[] = {kPlanPairs, 33, 15, 7};
  Plan best = {};
  double best_cost = 1e300;
  for (int i = 0; i < 10; ++i) {
    const int nt = kWidths[i];
    if (b_cols && nt % 32 != 0) continue;  // a CTA's half starts at a whole 16 bytes of the columns
    const double block = kBlockNs[i], epilogue = 600.0 + 9.5 * nt;
    for (int j = 0; j < 4; ++j) {
      const int parts = 1 << j, at_once = kAtOnce[j];
      const int slots = (nt + kChunk - 1) / kChunk * kChunk * kLanes * 4;
      if (parts > 1 && (parts > kblocks || (parts - 1) * slots > kRing)) break;
      Plan p;
      p.nt = nt;
      p.tiles_f = (int)((F + kTileF - 1) / kTileF);
      p.tiles_t = (int)((T + nt - 1) / nt);
      p.parts = parts;
      const int tiles = p.tiles_f * p.tiles_t;
      if (parts > 1 && tiles > at_once) break;
      p.clusters = min(tiles, at_once);
      const double tile = (double)((kblocks + parts - 1) / parts) * block + 400.0;
      const double cost = ((tiles + at_once - 1) / at_once) * fmax(tile, epilogue) + epilogue +
                          (parts > 1 ? 1500.0 + 4.0 * nt * parts : 0.0);
      if (cost < best_cost) {
        best_cost = cost;
        best = p;
      }
    }
  }
  return best;
}

inline int kblocks_of(long long bytes_or_rows, int per) { return (int)((bytes_or_rows + per - 1) / per); }

Plan plan_forward(int M, int N, int K, int in_type) {
  return make_plan(N, M, kblocks_of((long long)K * (in_type == DSPARK_E4M3 ? 1 : 2), 128), false);
}
Plan plan_dx(int M, int N, int K) { return make_plan(K, M, kblocks_of(N, 64), false); }
Plan plan_dw(int M, int N, int K) { return make_plan(K, N, kblocks_of(M, 64), true); }

// Row runs of dpre_kernel: enough CTAs for six on every SM, 32 rows or more each.
inline int dpre_runs(int M, int N) {
  const int cols = (N + 255) / 256;
  return max(1, min((M + 31) / 32, (12 * kPlanPairs + cols - 1) / cols));
}

template <bool F8, bool A_MN, bool B_MN, bool STAGED>
cudaError_t gemm_launch(Gemm g, const Plan& p, const CUtensorMap& ma, const CUtensorMap& mb, cudaStream_t s) {
  g.nt = p.nt;
  g.tiles_f = p.tiles_f;
  g.tiles_t = p.tiles_t;
  g.parts = p.parts;
  auto kern = linear_kernel<F8, A_MN, B_MN, STAGED>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess && p.parts > 4)  // clusters of 16 are past the portable size
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  return launch_early(kern, dim3((unsigned)(p.clusters * 2 * p.parts)), kThreads, kSmem, 2 * p.parts, s, ma, mb, g);
}

}  // namespace

size_t linear_scratch_bytes(int M, int N, int act) {
  const size_t dpre = act == DSPARK_ACT_NONE ? 0 : round_up((size_t)M * N * 2, 256);
  return dpre + round_up((size_t)dpre_runs(M, N) * N * sizeof(float), 256);
}

cudaError_t linear_launch(const LinearArgs& a, cudaStream_t s) {
  const bool f8 = a.in_type == DSPARK_E4M3;
  const int es = f8 ? 1 : 2;
  const Plan p = plan_forward(a.M, a.N, a.K, a.in_type);
  CUtensorMap ma, mb;
  if (!make_map(&ma, a.w, es, a.K, a.N, kLanes) || !make_map(&mb, a.x, es, a.K, a.M, p.nt / 2)) return cudaErrorInvalidValue;
  Gemm g = {};
  g.F = a.N;
  g.T = a.M;
  g.kblocks = kblocks_of((long long)a.K * es, 128);
  g.col_scale = a.x_scale;
  g.lane_scale = a.w_scale;
  g.bias = a.bias;
  g.residual = a.residual;
  g.out = a.y;
  g.pre = a.pre;
  g.out_type = a.out_type;
  g.act = a.act;
  g.status = a.status;
  const bool staged = g.out_type == DSPARK_BF16 && g.F % 8 == 0 && aligned16(g.out) && aligned16(g.residual) && aligned16(g.pre);
  if (f8)
    return staged ? gemm_launch<true, false, false, true>(g, p, ma, mb, s)
                  : gemm_launch<true, false, false, false>(g, p, ma, mb, s);
  return staged ? gemm_launch<false, false, false, true>(g, p, ma, mb, s)
                : gemm_launch<false, false, false, false>(g, p, ma, mb, s);
}

cudaError_t linear_grad_launch(const LinearGradArgs& a, cudaStream_t s) {
  const Plan px = plan_dx(a.M, a.N, a.K), pw = plan_dw(a.M, a.N, a.K);
  char* dpre_buf = a.scratch;
  float* partial = reinterpret_cast<float*>(dpre_buf + (a.act == DSPARK_ACT_NONE ? 0 : round_up((size_t)a.M * a.N * 2, 256)));
  const void* dpre = a.act == DSPARK_ACT_NONE ? a.dy : dpre_buf;
  cudaError_t e;
  const int runs = dpre_runs(a.M, a.N);
  if (a.act != DSPARK_ACT_NONE || a.dbias) {
    const int rows_per = (a.M + runs - 1) / runs;
    if (runs == 1) partial = a.dbias;  // one run's sums are the result
    auto kern = a.act == DSPARK_ACT_RELU   ? dpre_kernel<DSPARK_ACT_RELU>
                : a.act == DSPARK_ACT_SILU ? dpre_kernel<DSPARK_ACT_SILU>
                : a.act == DSPARK_ACT_GELU ? dpre_kernel<DSPARK_ACT_GELU>
                                           : dpre_kernel<DSPARK_ACT_NONE>;
    e = launch_early(kern, dim3((a.N + 255) / 256, runs), 256, 0, 1, s, a.dy, a.pre, a.M, a.N, rows_per, dpre_buf,
                     a.dbias ? partial : nullptr);
    if (e != cudaSuccess) return e;
  }
  CUtensorMap ma, mb;
  Gemm g = {};
  g.F = a.K;
  g.out_type = DSPARK_BF16;
  g.act = DSPARK_ACT_NONE;
  g.status = a.status;
  if (a.dx) {  // lanes k, columns m, contraction n
    if (!make_map(&ma, a.w, 2, a.K, a.N, 64) || !make_map(&mb, dpre, 2, a.N, a.M, px.nt / 2)) return cudaErrorInvalidValue;
    g.T = a.M;
    g.kblocks = kblocks_of(a.N, 64);
    g.out = a.dx;
    if ((e = gemm_launch<false, true, false, true>(g, px, ma, mb, s)) != cudaSuccess) return e;
  }
  if (a.dw) {  // lanes k, columns n, contraction m
    if (!make_map(&ma, a.x, 2, a.K, a.M, 64) || !make_map(&mb, dpre, 2, a.N, a.M, 64)) return cudaErrorInvalidValue;
    g.T = a.N;
    g.kblocks = kblocks_of(a.M, 64);
    g.out = a.dw;
    // dw takes nothing from dx: it starts on the SMs that dx leaves or never used, and
    // waits for dx before it ends (dx, dw and dbias at m5 n1456 k1640 22.7 us, one after
    // the other 24.6; m1341 n3808 k4984 110 and 116; m2048 n5120 k4096 142.5 and 143.9)
    if (a.dx) g.order = kBeside;
    if ((e = gemm_launch<false, true, true, true>(g, pw, ma, mb, s)) != cudaSuccess) return e;
  }
  // the sums need dpre_kernel's partial ones alone, which are complete where a product runs: they run
  // beside the last (dx, dw and dbias at m64 n1024 k1024 18.8 us, 22.4 before the products; m300
  // n2048 k2048 26.6 and 29.0)
  if (a.dbias && runs > 1) return column_sums_launch(partial, runs, a.N, a.dbias, s, a.dx || a.dw ? kBeside : kAfter);
  return cudaSuccess;
}

}  // namespace dspark
