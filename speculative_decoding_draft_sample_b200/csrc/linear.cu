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
// units (output tile, part of the contraction):
//   warp 0     TMA producer: 128-byte-wide boxes of this CTA's A and B into a ring
//              of stages; the bytes of both CTAs complete on the first one's barrier
//   warp 1     tensor-memory allocation and, in the first CTA, the single-thread
//              tcgen05.mma issuer
//   warps 2-17 epilogue of the previous unit meanwhile (two accumulators): a warp
//              reads its quarter of the lanes (hardware: warp index mod 4), the four
//              warps of a quarter take blocks of 32 columns in turn
// With fewer tiles than pairs the contraction is split: each part leaves its fp32
// sums in the workspace and the last to arrive adds them in order of the parts
// (the result does not depend on who that is) and finishes the tile.
// Every wait is bounded; a CTA that gives up reports DSPARK_STATUS_TIMEOUT.
#include "host.cuh"
#include "linear.cuh"
#include "norm.cuh"
#include "tcgen05.cuh"

namespace dspark {

namespace {

using namespace t5;

constexpr int kEpiWarps = 16;                  // four per quarter of the lanes, so that the latencies of a chunk overlap
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
  int nt;                   // columns per tile, a multiple of 16 (128 when B is column-contiguous)
  int tiles_f, tiles_t, splits;
  const float* col_scale;   // [T] or null
  const float* lane_scale;  // [F] or null
  const float* bias;        // [F] or null
  const void* residual;     // [T, F] or null
  void* out;                // [T, F]
  void* pre;                // [T, F] or null
  int out_type, act;
  int staged;               // bf16 rows of whole 16-byte vectors: through shared memory
  float* partial;           // [tile, split, 2, nt rounded up to 32, 128] (splits > 1)
  unsigned int* counter;    // [tile, CTA of the pair], zero at launch (splits > 1)
  Status* status;
};

// z / (1 + exp(-v)): silu with v = z, gelu's tanh form with v = 2 sqrt(2/pi) (z + 0.044715 z^3)
__device__ __forceinline__ float gate(float z, float v) { return __fdividef(z, 1.f + ex2(-v * kLog2e)); }

constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// act'(z); past |z| = 64 both gates are 0 or 1 exactly
__device__ __forceinline__ float activate_grad(float z, int act) {
  if (act == DSPARK_ACT_RELU) return z > 0.f ? 1.f : (z != z ? z : 0.f);
  z = z != z ? z : fminf(fmaxf(z, -64.f), 64.f);
  const float v = act == DSPARK_ACT_SILU ? z : kGelu2 * fmaf(0.044715f * z * z, z, z);
  const float dv = act == DSPARK_ACT_SILU ? 1.f : kGelu2 * fmaf(3.f * 0.044715f * z, z, 1.f);
  const float g = __fdividef(1.f, 1.f + ex2(-v * kLog2e));
  return g + z * g * (1.f - g) * dv;
}

__device__ __forceinline__ void activate32(float* v, int act) {
  if (act == DSPARK_ACT_RELU) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = v[j] < 0.f ? 0.f : v[j];  // NaN stays
  } else if (act == DSPARK_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = gate(v[j], v[j]);
  } else if (act == DSPARK_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = gate(v[j], kGelu2 * fmaf(0.044715f * v[j] * v[j], v[j], v[j]));
  }
}

// fp32 outputs (and 2-byte rows that are not whole 16-byte vectors): one lane's
// columns straight to memory, 32 neighbouring outputs per warp and store. All
// loads come before the first store: a load behind a store that might alias it
// waits for its turn. at: column 0; n columns.
template <int DT>
__device__ __forceinline__ void direct32(const Gemm& g, float* v, long long at, int n) {
  using T = typename Elem<DT>::T;
  if (g.pre) {
    T* p = static_cast<T*>(g.pre) + at;
#pragma unroll
    for (int j = 0; j < 32; ++j, p += g.F)
      if (j < n) *p = Elem<DT>::store_round(v[j]);
  }
  activate32(v, g.act);
  if (g.residual) {
    const T* p = static_cast<const T*>(g.residual) + at;
    T res[32];
#pragma unroll
    for (int j = 0; j < 32; ++j, p += g.F)
      if (j < n) res[j] = *p;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) v[j] += Elem<DT>::to_float(res[j]);
  }
  T* p = static_cast<T*>(g.out) + at;
#pragma unroll
  for (int j = 0; j < 32; ++j, p += g.F)
    if (j < n) *p = Elem<DT>::store_round(v[j]);
}

// bf16 outputs whose rows are whole 16-byte vectors go through shared memory: a
// lane holds features of many tokens, memory wants many features of one token.
// A warp's stage is its own (no barrier but the warp's): row r is token t0 + r,
// 32 features in four 16-byte vectors, vector q at q ^ (r / 2 % 4), so that eight
// rows of one vector and two rows of four both fall on all banks.
__device__ __forceinline__ uint32_t stage_at(int r, int q) { return r * 64 + ((q ^ ((r >> 1) & 3)) << 4); }

// Moves rows between a warp's stage and memory (p: token t0, the warp's first
// feature; nf features of the row remain): 8 rows x 64 bytes an instruction.
template <bool STORE>
__device__ __forceinline__ void move_rows(unsigned char* stage, uint16_t* p, int F, int nf, int rows, int lane) {
  const int q = lane & 3;
  if (q * 8 >= nf) return;
  p += (long long)(lane >> 2) * F + q * 8;
#pragma unroll
  for (int i = 0; i < kChunk / 8; ++i) {
    const int r = i * 8 + (lane >> 2);
    if (r < rows) {
      uint4* s = reinterpret_cast<uint4*>(stage + stage_at(r, q));
      uint4* d = reinterpret_cast<uint4*>(p + (long long)(i * 8) * F);
      if (STORE)
        *d = *s;
      else
        *s = *d;
    }
  }
}

// The work units of a pair, u = pair, pair + pairs, ...: unit u is part
// u % splits of tile u / splits, and tiles run over the columns first, so that
// pairs working at the same time share their rows of A. Steps by additions: a
// unit of a short contraction lasts less than four divisions in a row.
struct Units {
  int u, left, sp, tt, tf;
  int dsp, dtt, dtf, splits, tiles_t;
  __device__ __forceinline__ Units(const Gemm& g, int pair, int pairs)
      : u(pair), splits(g.splits), tiles_t(g.tiles_t) {
    const int units = g.tiles_f * g.tiles_t * g.splits;
    left = units > pair ? (units - pair + pairs - 1) / pairs : 0;
    sp = pair % splits;
    tt = pair / splits % tiles_t;
    tf = pair / splits / tiles_t;
    dsp = pairs % splits;
    dtt = pairs / splits % tiles_t;
    dtf = pairs / splits / tiles_t;
  }
  __device__ __forceinline__ void next() {
    --left;
    sp += dsp;
    tt += dtt;
    tf += dtf;
    if (sp >= splits) {
      sp -= splits;
      ++tt;
    }
    if (tt >= tiles_t) {
      tt -= tiles_t;
      ++tf;
    }
  }
  // the part's blocks of the contraction
  __device__ __forceinline__ void blocks(const Gemm& g, int& k0, int& k1) const {
    k0 = 0;
    k1 = g.kblocks;
    if (splits > 1) {
      k0 = (int)((long long)g.kblocks * sp / splits);
      k1 = (int)((long long)g.kblocks * (sp + 1) / splits);
    }
  }
};

__device__ __forceinline__ void epi_bar() { asm volatile("bar.sync 1, 512;" ::: "memory"); }

// A_MN / B_MN: the operand is contiguous along lanes / columns, not along the contraction.
template <bool F8, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, Gemm g) {
  extern __shared__ __align__(1024) unsigned char smem[];
  if (su32(smem) & 1023u) {  // 128-byte-swizzled tiles need 1024-byte alignment (the same offset in every CTA)
    if (threadIdx.x == 0) report(g.status, DSPARK_STATUS_INTERNAL, 0);
    return;
  }
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* last_flag = abort_flag + 1;
  volatile int* dead = abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cta_rank();
  const int nh = g.nt / 2;  // columns of B in this CTA
  const int stage_bytes = kABytes + nh * 128;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int stages = min(kMaxStages, kRing / stage_bytes);
  Units w(g, pair, pairs);

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

  // The producer and the issuer are one thread each, whose loop has to keep up
  // with a block of 512 tensor-core cycles: stages and phases are counted, not
  // divided, and addresses and descriptors advance by additions (a loop that
  // computed them anew took 730 cycles a block).
  if (warp == 0) {
    if (lane == 0) {
      const uint32_t smem0 = su32(smem), full0 = map_rank(su32(full), 0);
      int s = 0, issued = 0;
      uint32_t ph = 1;
      for (; w.left > 0 && !*dead; w.next()) {
        const int f0 = w.tf * kTileF + rank * kLanes, t0 = w.tt * g.nt + rank * nh;
        int k0, k1;
        w.blocks(g, k0, k1);
        int kx = k0 * (F8 ? 128 : 64);
        for (int kb = k0; kb < k1; ++kb, kx += F8 ? 128 : 64) {
          if (!mbar_wait(&empty[s], ph)) {
            if (!*dead) report_wait(g.status, kWhereEmpty, 0);
            *dead = 1;
            break;
          }
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
            for (int q = 0; q < nh / 64; ++q) tma_load_2d(b + q * kBoxBytes, &map_b, t0 + q * 64, kx, bar);
          } else {
            tma_load_2d(b, &map_b, kx, t0, bar);
          }
          ++issued;
          if (++s == stages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (*dead && rank == 0)  // let issued loads of both CTAs land before the pair winds down (below)
        for (int q = max(0, issued - stages); q < issued; ++q) mbar_wait(&full[q % stages], (q / stages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
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
      for (; w.left > 0 && !*dead; w.next()) {
        int k0, k1;
        w.blocks(g, k0, k1);
        if (!mbar_wait(&acc_empty[buf], aph)) {
          if (!*dead) report_wait(g.status, kWhereAccEmpty, 0);
          *dead = 1;
          break;
        }
        fence_after();
        const uint32_t d = tmem + buf * kMaxCols;
        uint32_t acc = 0;
        for (int kb = k0; kb < k1; ++kb) {
          if (!mbar_wait(&full[s], ph)) {
            if (!*dead) report_wait(g.status, kWhereFull, 0);
            *dead = 1;
            break;
          }
          fence_after();
#pragma unroll
          for (int q = 0; q < 4; ++q) {  // 32 bytes of the contraction (or 16 rows of it) each
            mma<F8>(d, da + q * step_a, db + q * step_b, idesc, acc);
            acc = 1;
          }
          mma_commit(&empty[s]);
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
        if (*dead) break;
        mma_commit(&acc_full[buf]);
        buf ^= 1;
        if (buf == 0) aph ^= 1;
      }
      if (*dead && done > 0)  // MMAs complete in order: after the last commit tensor memory is quiet
        mbar_wait(&empty[(done - 1) % stages], ((done - 1) / stages) & 1);
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3, group = (warp - 2) >> 2;
    const int ln = quarter * 32 + lane;    // lane of this CTA's part of the tile
    const uint32_t acc_free = map_rank(su32(acc_empty), 0);
    unsigned char* stage = smem + kOffStage + (warp - 2) * kStageBytes;
    const uint32_t mat = su32(stage) + stage_at(lane & 7, lane >> 3);  // + 512 for the next 8 columns
    // the features whose values this thread holds: one lane's, or four rows of its fragments
    const int nrow = g.staged ? 4 : 1, row0 = g.staged ? quarter * 32 + (lane >> 2) : ln;
    float ls[4], bias[4];

    // 32 columns from c of the tile to the outputs; cscale: lane j's is column j's scale
    auto finish = [&](float* v, int f0, int t0, int c, float cscale) {
      if (!g.staged) {
        if (g.lane_scale) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] *= ls[0] * __shfl_sync(0xffffffffu, cscale, j);
        }
        if (g.bias) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] += bias[0];
        }
        const int n = f0 + ln < g.F ? min(min(kChunk, g.nt - c), g.T - t0 - c) : 0;
        const long long at = (long long)(t0 + c) * g.F + f0 + ln;
        if (g.out_type == DSPARK_F32)
          direct32<DSPARK_F32>(g, v, at, n);
        else
          direct32<DSPARK_BF16>(g, v, at, n);
        return;
      }
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
        for (int j = 0; j < 32; ++j) v[j] += bias[2 * (j >> 4) + ((j >> 1) & 1)];
      }
      const int rows = min(min(kChunk, g.nt - c), g.T - t0 - c), fw = f0 + quarter * 32;
      const long long at = (long long)(t0 + c) * g.F + fw;
      auto put = [&](void* p) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float* a = v + 16 * (i >> 1) + 4 * k + 2 * (i & 1);
            w[i] = pack_bf16x2(a[0], a[1]);
          }
          store_matrix_t(mat + k * 512, w);
        }
        __syncwarp();
        move_rows<true>(stage, static_cast<uint16_t*>(p) + at, g.F, g.F - fw, rows, lane);
        __syncwarp();  // the stage is free again
      };
      if (g.pre) put(g.pre);
      activate32(v, g.act);
      if (g.residual) {
        move_rows<false>(stage, const_cast<uint16_t*>(static_cast<const uint16_t*>(g.residual)) + at, g.F, g.F - fw, rows, lane);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
          load_matrix_t(mat + k * 512, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float* a = v + 16 * (i >> 1) + 4 * k + 2 * (i & 1);
            a[0] += __uint_as_float(w[i] << 16);
            a[1] += __uint_as_float(w[i] & 0xffff0000u);
          }
        }
        __syncwarp();
      }
      put(g.out);
    };

    // A warp whose wait gives up goes on without its work: the barriers of a
    // split contraction expect every warp.
    uint32_t buf = 0, aph = 0;
    for (; w.left > 0; w.next()) {
      const int f0 = w.tf * kTileF + rank * kLanes, t0 = w.tt * g.nt;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int f = f0 + row0 + 8 * i;
        const bool in = i < nrow && f < g.F;
        ls[i] = g.lane_scale && in ? __ldg(g.lane_scale + f) : 0.f;
        bias[i] = g.bias && in ? __ldg(g.bias + f) : 0.f;
      }
      bool ok = !*dead;
      if (ok && !mbar_wait(&acc_full[buf], aph)) {
        ok = false;
        if (!*dead) report_wait(g.status, kWhereAccFull, 0);
        *dead = 1;
      }
      ok = __all_sync(0xffffffffu, ok);
      fence_after();
      const uint32_t src = tmem + buf * kMaxCols + ((uint32_t)(quarter * 32) << 16);
      // partial sums in the threads' own order: [tile, split, CTA, chunk, value, lane]
      const int chunks = (g.nt + kChunk - 1) / kChunk, tile = w.tf * g.tiles_t + w.tt;
      float* part = g.partial + ((size_t)tile * g.splits * 2 + rank) * chunks * (kChunk * 128) + ln;
      const size_t part_split = (size_t)2 * chunks * (kChunk * 128);
      const int c1 = ok ? min(g.nt, g.T - t0) : 0;
      for (int c = group * kChunk; c < c1; c += kEpiWarps / 4 * kChunk) {
        float v[32];
        const float cscale = g.col_scale && t0 + c + lane < g.T ? __ldg(g.col_scale + t0 + c + lane) : 0.f;
        if (g.staged)
          tmem_ld_frags(src + c, v);
        else
          tmem_ld_lanes(src + c, v);
        if (c + kEpiWarps / 4 * kChunk >= c1) {  // the warp's last chunk: its part of the accumulator is free
          fence_before();
          if (lane == 0) mbar_arrive_relaxed(acc_free + 8 * buf);
        }
        if (g.splits == 1) {
          finish(v, f0, t0, c, cscale);
        } else {
          float* p = part + w.sp * part_split + (size_t)(c / kChunk) * (kChunk * 128);
#pragma unroll
          for (int j = 0; j < 32; ++j) p[j * 128] = v[j];
        }
      }
      if (group * kChunk >= c1 && lane == 0) mbar_arrive_relaxed(acc_free + 8 * buf);  // nothing to read
      if (g.splits > 1) {
        __threadfence();
        epi_bar();
        if (tid == 64) *last_flag = atomicAdd(&g.counter[2 * tile + rank], 1u) == (unsigned)g.splits - 1;
        epi_bar();
        if (*(volatile int*)last_flag) {
          __threadfence();
          for (int c = group * kChunk; c < c1; c += kEpiWarps / 4 * kChunk) {
            const float cscale = g.col_scale && t0 + c + lane < g.T ? __ldg(g.col_scale + t0 + c + lane) : 0.f;
            const float* p = part + (size_t)(c / kChunk) * (kChunk * 128);
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.f;
            for (int q = 0; q < g.splits; ++q, p += part_split)
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] += __ldcg(p + j * 128);
            finish(v, f0, t0, c, cscale);
          }
        }
      }
      buf ^= 1;
      if (buf == 0) aph ^= 1;
    }
  }
  fence_before();
  cluster_sync();  // neither CTA leaves while the other's arrivals or loads may still reach it
  fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// dpre = round_bf16(dy act'(pre)) (the tensor cores take bf16 operands; the
// rounding is half a bf16 step of each factor, as in the bf16 result) and
// per-CTA column sums of the unrounded values. A CTA takes 256 columns and a
// contiguous run of rows, 8 rows at a time.
constexpr int kDpreRows = 8;

__global__ void __launch_bounds__(256) dpre_kernel(const void* dy, const void* pre, int M, int N, int act, int rows_per,
                                                   void* dpre, float* partial) {
  __shared__ float part[kDpreRows][256 + 8];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int n0 = blockIdx.x * 256 + lane * 8;
  const int m1 = min(M, (int)(blockIdx.y + 1) * rows_per);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (n0 < N) {
    for (int m = blockIdx.y * rows_per + row; m < m1; m += kDpreRows) {
      const size_t at = ((size_t)m * N + n0) * 2;
      float d[8];
      Vec16<DSPARK_BF16>::load(static_cast<const char*>(dy) + at, d);
      if (act != DSPARK_ACT_NONE) {
        float z[8];
        Vec16<DSPARK_BF16>::load(static_cast<const char*>(pre) + at, z);
        alignas(16) uint16_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          d[e] *= activate_grad(z[e], act);
          o[e] = Elem<DSPARK_BF16>::store_round(d[e]);
        }
        *reinterpret_cast<uint4*>(static_cast<char*>(dpre) + at) = *reinterpret_cast<const uint4*>(o);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += d[e];
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
  int nt, tiles_f, tiles_t, splits;
  size_t partial_bytes() const {
    return splits > 1 ? (size_t)tiles_f * tiles_t * splits * round_up(nt, kChunk) * kTileF * sizeof(float) : 0;
  }
  size_t counter_bytes() const { return splits > 1 ? round_up((size_t)tiles_f * tiles_t * 2 * sizeof(unsigned int), 256) : 0; }
  size_t bytes() const { return counter_bytes() + round_up(partial_bytes(), 256); }
};

// The column width and the split of the contraction with the least time by a
// count of cycles: a 128-byte block of a stage costs its bytes at 64 a cycle or
// its matrix instructions (nt / 2 cycles each), whichever is more; a unit adds
// a fixed start and end.
Plan make_plan(long long F, long long T, int kblocks, int min_nt) {
  Plan best = {};
  double best_cost = 1e300;
  for (int nt = min_nt; nt <= kMaxCols; nt *= 2) {
    Plan p;
    p.nt = nt;
    p.tiles_f = (int)((F + kTileF - 1) / kTileF);
    p.tiles_t = (int)((T + nt - 1) / nt);
    const long long tiles = (long long)p.tiles_f * p.tiles_t;
    p.splits = (int)(tiles < kPlanPairs ? kPlanPairs / tiles : 1);
    if (p.splits > kblocks / 4) p.splits = kblocks / 4;
    if (p.splits < 1) p.splits = 1;
    const long long waves = (tiles * p.splits + kPlanPairs - 1) / kPlanPairs;
    const double block = fmax((kABytes + nt * 64) / 64.0, 2.0 * nt);
    const double unit = (double)((kblocks + p.splits - 1) / p.splits) * block + 1500 + 8.0 * nt * (p.splits > 1 ? 2 : 1);
    const double cost = waves * unit;
    if (cost < best_cost) {
      best_cost = cost;
      best = p;
    }
  }
  return best;
}

inline int kblocks_of(long long bytes_or_rows, int per) { return (int)((bytes_or_rows + per - 1) / per); }

Plan plan_forward(int M, int N, int K, int in_type) {
  return make_plan(N, M, in_type == DSPARK_E4M3 ? kblocks_of(K, 128) : kblocks_of(K, 64), 16);
}
Plan plan_dx(int M, int N, int K) { return make_plan(K, M, kblocks_of(N, 64), 16); }
Plan plan_dw(int M, int N, int K) { return make_plan(K, N, kblocks_of(M, 64), 128); }

// Row runs of dpre_kernel: enough CTAs for two on every SM, 64 rows or more each.
inline int dpre_runs(int M, int N) {
  const int cols = (N + 255) / 256;
  return max(1, min((M + 63) / 64, (4 * kPlanPairs + cols - 1) / cols));
}

template <bool F8, bool A_MN, bool B_MN>
cudaError_t gemm_launch(Gemm g, const Plan& p, const CUtensorMap& ma, const CUtensorMap& mb, char* scratch, int num_sms,
                        cudaStream_t s) {
  g.nt = p.nt;
  g.tiles_f = p.tiles_f;
  g.tiles_t = p.tiles_t;
  g.splits = p.splits;
  g.staged = g.out_type == DSPARK_BF16 && g.F % 8 == 0 && aligned16(g.out) && aligned16(g.residual) && aligned16(g.pre);
  cudaError_t e;
  if (p.splits > 1) {
    g.counter = reinterpret_cast<unsigned int*>(scratch);
    g.partial = reinterpret_cast<float*>(scratch + p.counter_bytes());
    e = cudaMemsetAsync(g.counter, 0, p.counter_bytes(), s);
    if (e != cudaSuccess) return e;
  }
  auto kern = linear_kernel<F8, A_MN, B_MN>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const long long units = (long long)p.tiles_f * p.tiles_t * p.splits;
  kern<<<2 * (unsigned)min(units, (long long)num_sms / 2), kThreads, kSmem, s>>>(ma, mb, g);
  return cudaGetLastError();
}

}  // namespace

size_t linear_scratch_bytes(int M, int N, int K, int in_type) {
  size_t n = plan_forward(M, N, K, in_type).bytes();
  if (in_type == DSPARK_BF16) {
    const size_t split = max(plan_dx(M, N, K).bytes(), plan_dw(M, N, K).bytes());
    const size_t grad = split + round_up((size_t)M * N * 2, 256) + round_up((size_t)dpre_runs(M, N) * N * sizeof(float), 256);
    if (grad > n) n = grad;
  }
  return n;
}

cudaError_t linear_launch(const LinearArgs& a, int num_sms, cudaStream_t s) {
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
  return f8 ? gemm_launch<true, false, false>(g, p, ma, mb, a.scratch, num_sms, s)
            : gemm_launch<false, false, false>(g, p, ma, mb, a.scratch, num_sms, s);
}

cudaError_t linear_grad_launch(const LinearGradArgs& a, int num_sms, cudaStream_t s) {
  const Plan px = plan_dx(a.M, a.N, a.K), pw = plan_dw(a.M, a.N, a.K);
  char* split = a.scratch;
  char* dpre_buf = split + max(px.bytes(), pw.bytes());
  float* partial = reinterpret_cast<float*>(dpre_buf + round_up((size_t)a.M * a.N * 2, 256));
  const void* dpre = a.act == DSPARK_ACT_NONE ? a.dy : dpre_buf;
  cudaError_t e;
  if (a.act != DSPARK_ACT_NONE || a.dbias) {
    const int runs = dpre_runs(a.M, a.N);
    const int rows_per = (a.M + runs - 1) / runs;
    dpre_kernel<<<dim3((a.N + 255) / 256, runs), 256, 0, s>>>(a.dy, a.pre, a.M, a.N, a.act, rows_per, dpre_buf,
                                                              a.dbias ? partial : nullptr);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (a.dbias && (e = column_sums_launch(partial, runs, a.N, a.dbias, s)) != cudaSuccess) return e;
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
    if ((e = gemm_launch<false, true, false>(g, px, ma, mb, split, num_sms, s)) != cudaSuccess) return e;
  }
  if (a.dw) {  // lanes k, columns n, contraction m
    if (!make_map(&ma, a.x, 2, a.K, a.M, 64) || !make_map(&mb, dpre, 2, a.N, a.M, 64)) return cudaErrorInvalidValue;
    g.T = a.N;
    g.kblocks = kblocks_of(a.M, 64);
    g.out = a.dw;
    if ((e = gemm_launch<false, true, true>(g, pw, ma, mb, split, num_sms, s)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace dspark
