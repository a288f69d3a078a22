// Product of two 4-bit microscaled matrices, D[m][n] = sum_k A[m][k] B[n][k], both MXFP4 or both
// NVFP4 (codes and scales row-major, as the quantisers leave them), FP32 accumulation, one
// rounding to BF16, FP16 or FP32: a W4A4 projection with A the activations and B the weights.
//
// tcgen05.mma block-scaled over CTA pairs, 256 x 256 tiles; kind::mxf4 (E2M1, one UE8M0 scale
// per 32) or kind::mxf4nvf4 (E2M1, one E4M3 scale per 16).  The scales multiply inside the
// MMA; NVFP4's two tensor scales multiply the accumulator.
//
// B's rows (the weights' features) are the tensor core's M and A's rows (tokens) its N, which
// may be any multiple of 32 up to 256: one token costs an N of 32, and the kernel streams weights.
//
// Scales.  The tensor core wants them in TMEM: the scales of operand row m at lane m % 32 (in
// all four lane quarters), column m / 32, 32 bits per row and K group.  Four warps of each CTA
// read them from the row-major bytes that TMA brought (16 bytes per row and K step) and store
// them with tcgen05.st, each its lane quarter: a copy on the tensor pipe would wait for
// the MMAs there.  Each CTA needs the scales of its own 128 M rows and of all N rows.  Bytes
// past a row's last scale are filled with zeros by TMA, so that what lies behind them in memory
// (a NaN byte times a zero code would be NaN) does not matter.
//
// Few tiles.  A decoding step has one row block and few feature tiles (20 for 5120 features), too
// few pairs to draw weights at the memory's rate.  Then a cluster of S pairs shares a tile: each
// multiplies its stretch of K, and the first pair adds the others' sums, copied into its shared
// memory, in their order (the result does not depend on timing).
//
// A CTA (768 threads): warp 0 loads (a ring of 5 stages of 38 KB: 256 K values of 128 B rows
// and of half of the A rows, and their scales), warp 1 of the leading CTA issues the MMAs, warp
// 3 owns TMEM, warps 4..7 move scales, warps 8..23 store results.  One accumulator of 256
// columns (the scales of five stages take the other half of TMEM): the storing warps read it
// into registers and release it before they convert and store.
//
// What bounds it.  16384 x 5120 x 5120: MXFP4 174 us (4.9 PFLOP/s), NVFP4 187; the tensor pipe is
// active 60% of the cycles, the MMAs wait for the accumulator's drain between tiles and for
// stages (a ring of four: 8% slower); in a long loop the power limit sets the clock (1.5 GHz, 202 and
// 217 us).  A second set of scale warps, results turned in shared memory, sleeping waits: each was
// slower.  One token, 5120 x 5120: 6.0 us with the weights in L2, 7.6 without, of which a launch
// with one K step is 3.7.
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "../../include/beam_moe.h"
#include "cta_pair.cuh"
#include "internal.h"
#include "overlap.h"

namespace beam {

namespace {

__device__ uint32_t g_fp4_err;  // error bits of this device's 4-bit products

constexpr int F4_BK = 256;                      // K values of a stage: one 128-byte line of codes
constexpr int F4_STAGES = 5;
constexpr int F4_CODES = 128 * 128;             // 16 KB: codes of 128 rows
constexpr int F4_OFF_N = F4_CODES;              // N-side codes
constexpr int F4_OFF_SFM = 2 * F4_CODES;        // scales of this CTA's 128 M rows
constexpr int F4_OFF_SFN = F4_OFF_SFM + 128 * 16;
constexpr int F4_STAGE = F4_OFF_SFN + 256 * 16;
static_assert(F4_STAGE % 1024 == 0, "swizzled lines start on 1 KB boundaries");
constexpr int F4_TILE = 256;
constexpr int F4_PANEL = 8;                     // row blocks of A that share B in turn
constexpr int F4_SF_COL = 256;                  // TMEM columns of the stages' scales
constexpr int F4_SF_STAGE = 48;                 // M: 4 columns per K group, then N: 8 per K group
constexpr int F4_SF_N = 16;
static_assert(F4_SF_COL + F4_STAGES * F4_SF_STAGE <= 512, "scales fit in TMEM");
constexpr int F4_MAX_SPLIT = 4;                 // pairs that share a tile
constexpr int F4_MAX_SHARE = 1 << 20;           // stages of a pair's share: 0.3 us each, far below the wait limit
constexpr int F4_SUM_ROWS = 64;                 // rows of sums that a shared tile's first pair can receive
constexpr int F4_FIRST_SF = 4, F4_FIRST_EPI = 8, F4_EPI_WARPS = 16;
constexpr int F4_THREADS = 32 * (F4_FIRST_EPI + F4_EPI_WARPS);

struct Fp4Args {
  int m, n, k;             // D is [m][n]
  int blocks, height;      // A's rows in equal blocks, their height a multiple of 32 up to 256
  int split;               // pairs that share a tile (1: each pair its own tiles)
  const float* alpha_a;    // tensor scales, or nullptr
  const float* alpha_b;
  void* out;
  int64_t ldo;
};

struct __align__(16) Fp4Tail {
  uint64_t full[F4_STAGES];      // this CTA's operands and scales have landed
  uint64_t empty[F4_STAGES];
  uint64_t sf_full[F4_STAGES];   // leader: both CTAs' scales are in TMEM (their operands have landed)
  uint64_t acc_full;
  uint64_t acc_empty;            // leader
  uint64_t drain;
  uint64_t sums_full;            // shared tiles: the other pairs' sums have come
  uint32_t tmem_base;
  int abort_flag;
  uint32_t progress;             // stages loaded
  alignas(16) float sums[F4_SUM_ROWS * 128];  // shared tiles: received sums
};
constexpr size_t kFp4Smem = static_cast<size_t>(F4_STAGES) * F4_STAGE + sizeof(Fp4Tail) + 1024;
static_assert(kFp4Smem <= 227 * 1024, "shared memory of one CTA");

struct Fp4Tile {
  int f0;          // first feature (row of B)
  int r0, r_end;   // rows of A
  int n;           // their number rounded up to 32
};

__device__ __forceinline__ Fp4Tile fp4_tile(const Fp4Args& a, int id) {
  Fp4Tile t;
  const int ft = (a.n + F4_TILE - 1) / F4_TILE;
  const int panel = id / (F4_PANEL * ft);
  const int rest = id - panel * F4_PANEL * ft;
  const int wide = min(F4_PANEL, a.blocks - panel * F4_PANEL);
  t.f0 = rest / wide * F4_TILE;
  const int block = panel * F4_PANEL + rest % wide;
  t.r0 = block * a.height;
  t.r_end = min(a.m, t.r0 + a.height);
  t.n = max(32, (t.r_end - t.r0 + 31) & ~31);
  return t;
}

// The two tensor scales: `scale` is their product, and `first` 1, wherever the product is a normal
// number.  Where it is not (1e-23 and 1e-23, say, with sums around 1e10) a sum takes the larger scale
// first and then the smaller, which leaves the normal range only where the result does.
struct TensorScales {
  float first, scale;
};
__device__ __forceinline__ TensorScales tensor_scales(const float* alpha_a, const float* alpha_b) {
  const float a = alpha_a ? __ldcg(alpha_a) : 1.0f, b = alpha_b ? __ldcg(alpha_b) : 1.0f;
  const float p = a * b;
  const bool plain = (fabsf(p) >= 0x1p-126f && fabsf(p) < INFINITY) || a == 0.0f || b == 0.0f ||
                     !(fabsf(a) < INFINITY) || !(fabsf(b) < INFINITY);
  if (plain) return {1.0f, p};
  return fabsf(a) >= fabsf(b) ? TensorScales{a, b} : TensorScales{b, a};
}

template <int FORMAT>
__device__ __forceinline__ void tc_mma_fp4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint32_t sfa, uint32_t sfb, uint32_t accumulate, uint32_t leader) {
  if constexpr (FORMAT == BEAM_MOE_FP4_MX)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(leader)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(leader)
        : "memory");
}

// Boxes: 128 rows of B; half a block's and a whole block's rows of A (the last block is shorter:
// what its boxes bring of later rows, or zeros, feeds accumulator columns that are not stored).
struct Fp4Maps {
  CUtensorMap m_codes, n_codes, m_sf, n_sf;
};

template <int FORMAT, int OUT, bool kSplit>
__global__ void __launch_bounds__(F4_THREADS, 1)
    gemm_fp4_kernel(const Fp4Args args, const __grid_constant__ Fp4Maps maps) {
  constexpr bool kMx = FORMAT == BEAM_MOE_FP4_MX;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Fp4Tail* tail = reinterpret_cast<Fp4Tail*>(smem + F4_STAGES * F4_STAGE);
  volatile int* abort_flag = &tail->abort_flag;
  volatile uint32_t* progress = &tail->progress;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t cluster_rank = cluster_cta_rank();
  const uint32_t rank = cluster_rank & 1;                        // in the pair
  const uint32_t first = kSplit ? cluster_rank & ~1u : 0u;       // the pair's leading CTA
  const int pair = kSplit ? static_cast<int>(cluster_rank >> 1) : 0;

  if (threadIdx.x == 0) {
    prefetch_tmap(&maps.m_codes);
    prefetch_tmap(&maps.n_codes);
    prefetch_tmap(&maps.m_sf);
    prefetch_tmap(&maps.n_sf);
    for (int i = 0; i < F4_STAGES; ++i) {
      mbar_init(&tail->full[i], 1);
      mbar_init(&tail->empty[i], 1);
      mbar_init(&tail->sf_full[i], 8);
    }
    mbar_init(&tail->acc_full, 1);
    mbar_init(&tail->acc_empty, 2 * F4_EPI_WARPS);
    mbar_init(&tail->drain, 1);
    mbar_init(&tail->sums_full, 1);
    if (kSplit && pair == 0)
      mbar_arrive_expect_tx(&tail->sums_full, static_cast<uint32_t>((args.split - 1) * args.m) * 512);
    tail->abort_flag = 0;
    tail->progress = 0;
    fence_mbar_init();
  }
  if (warp == 3) {
    tmem_alloc_pair(&tail->tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers are set before anyone arrives at them
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = tail->tmem_base;
  const int total = args.blocks * ((args.n + F4_TILE - 1) / F4_TILE);
  const int all_steps = (args.k + F4_BK - 1) / F4_BK;
  // this pair's tiles and K steps: every tile_stride-th tile, or one tile and a share of its steps
  const int first_tile = kSplit ? static_cast<int>(blockIdx.x) / (2 * args.split) : blockIdx.x >> 1;
  const int tile_stride = kSplit ? total : gridDim.x >> 1;
  const int step0 = kSplit ? all_steps * pair / args.split : 0;
  const int step1 = kSplit ? all_steps * (pair + 1) / args.split : all_steps;

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    int stage = 0;
    uint32_t phase = 0, loaded = 0;
    bool ok = true;
    const uint32_t code_bytes = F4_CODES + static_cast<uint32_t>(args.height) * (128 / 2);
    const uint32_t sf_bytes = 128 * 16 + static_cast<uint32_t>(args.height) * 16;
    for (int id = first_tile; id < total && ok; id += tile_stride) {
      const Fp4Tile t = fp4_tile(args, id);
      const int half = t.n >> 1;
      const int f0 = t.f0 + static_cast<int>(rank) * 128, r0 = t.r0 + static_cast<int>(rank) * half;
      for (int i = step0; i < step1; ++i) {
        ok = __all_sync(0xffffffffu, pair_wait(&tail->empty[stage], phase ^ 1, abort_flag));
        if (!ok) break;
        ++loaded;
        if (elect_one()) {
          *progress = loaded;
          uint8_t* s = smem + stage * F4_STAGE;
          uint64_t* bar = &tail->full[stage];
          // 16 scale bytes of a row: this K step's (NVFP4), or those of an even step and the next,
          // which finds them in the scale warps' registers
          const bool scales = !kMx || (i & 1) == 0 || i == step0;
          mbar_arrive_expect_tx(bar, code_bytes + (scales ? sf_bytes : 0));
          tma_load_2d(s, &maps.m_codes, bar, i * 128, f0);
          tma_load_2d(s + F4_OFF_N, &maps.n_codes, bar, i * 128, r0);
          if (scales) {
            const int sx = kMx ? (i >> 1) * 16 : i * 16;
            tma_load_2d(s + F4_OFF_SFM, &maps.m_sf, bar, sx, f0);
            tma_load_2d(s + F4_OFF_SFN, &maps.n_sf, bar, sx, t.r0);
          }
        }
        __syncwarp();
        if (++stage == F4_STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) {  // the copies still in flight land long before this
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    if (rank == 0) {
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, ready = false;
      const uint32_t leader = elect_one() ? 1u : 0u;
      // E2M1 operands, E4M3 or UE8M0 scales, K-major, M = 256
      const uint32_t idesc0 = (1u << 7) | (1u << 10) | ((kMx ? 1u : 0u) << 23) | ((F4_TILE >> 4) << 24);
      const uint64_t da0 = sdesc_k_sw128(smem_u32(smem)), db0 = sdesc_k_sw128(smem_u32(smem) + F4_OFF_N);
      for (int id = first_tile; id < total && ok; id += tile_stride) {
        const Fp4Tile t = fp4_tile(args, id);
        ok = __all_sync(0xffffffffu, pair_wait(&tail->acc_empty, acc_phase ^ 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const uint32_t idesc = idesc0 | (static_cast<uint32_t>(t.n >> 3) << 17);
        for (int i = step0; i < step1; ++i) {
          if (!ready) {
            ok = __all_sync(0xffffffffu, pair_wait(&tail->sf_full[stage], phase, abort_flag));
            if (!ok) break;
          }
          tc_fence_after();
          // look at the next stage's barrier while this stage's MMAs go out
          const int next = stage + 1 == F4_STAGES ? 0 : stage + 1;
          const uint32_t next_phase = phase ^ (next == 0 ? 1u : 0u);
          const bool next_ready = mbar_test(&tail->sf_full[next], next_phase);
          const uint64_t da = da0 + static_cast<uint64_t>(stage * (F4_STAGE / 16));
          const uint64_t db = db0 + static_cast<uint64_t>(stage * (F4_STAGE / 16));
          const uint32_t sf = tmem + F4_SF_COL + stage * F4_SF_STAGE;
          const int left = args.k - i * F4_BK;
#pragma unroll
          for (int j = 0; j < F4_BK / 64; ++j) {
            if (j * 64 >= left) break;
            // MXFP4: a 32-bit cell holds the scales of 128 values; the descriptor picks the half
            const int group = kMx ? j >> 1 : j;
            const uint32_t half = kMx ? static_cast<uint32_t>(j & 1) * 2 : 0u;
            tc_mma_fp4_pair<FORMAT>(tmem, da + j * 2, db + j * 2, idesc | (half << 29) | (half << 4), sf + group * 4,
                                    sf + F4_SF_N + group * 8, ((i - step0) | j) != 0 ? 1u : 0u, leader);
          }
          tc_commit_pair(&tail->empty[stage], leader, first);
          stage = next;
          phase = next_phase;
          ready = __all_sync(0xffffffffu, next_ready);
        }
        if (!ok) break;
        tc_commit_pair(&tail->acc_full, leader, first);
        acc_phase ^= 1;
      }
      if (!ok) {  // nothing may read shared memory or write TMEM after the CTAs are gone
        tc_commit_pair(&tail->drain, leader, first);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&tail->drain, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else if (warp >= F4_FIRST_SF && warp < F4_FIRST_EPI) {
    // ------------------------------------------------------------ scales -> TMEM
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int id = first_tile; id < total && ok; id += tile_stride) {
      uint4 held[12];  // MXFP4: the scales of an even step and the next
      for (int i = step0; i < step1; ++i) {
        ok = __all_sync(0xffffffffu, pair_wait(&tail->full[stage], phase, abort_flag));
        if (!ok) break;
        const uint8_t* sm = smem + stage * F4_STAGE + F4_OFF_SFM + lane * 16;
        const uint8_t* sn = smem + stage * F4_STAGE + F4_OFF_SFN + lane * 16;
        const uint32_t col = t_lane + F4_SF_COL + stage * F4_SF_STAGE;
        // lane l takes rows l, l + 32, ...: row l + 32 q goes to column q (and 4 more for N rows
        // from 128 on) of its K group
        if constexpr (kMx) {
          if ((i & 1) == 0 || i == step0) {
#pragma unroll
            for (int q = 0; q < 4; ++q) held[q] = *reinterpret_cast<const uint4*>(sm + q * 512);
#pragma unroll
            for (int q = 0; q < 8; ++q) held[4 + q] = *reinterpret_cast<const uint4*>(sn + q * 512);
          }
          const bool upper = (i & 1) != 0;
          uint32_t r[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            r[q] = upper ? held[q].z : held[q].x;
            r[4 + q] = upper ? held[q].w : held[q].y;
          }
          tmem_st_32x32b_x8(col, r);
          uint32_t w[16];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            w[q] = upper ? held[4 + q].z : held[4 + q].x;
            w[8 + q] = upper ? held[4 + q].w : held[4 + q].y;
          }
          tmem_st_32x32b_x16(col + F4_SF_N, w);
        } else {
          // all loads first: the stores of one part would hold up the next part's loads
          uint4 v[12];
#pragma unroll
          for (int q = 0; q < 12; ++q)
            v[q] = *reinterpret_cast<const uint4*>(q < 4 ? sm + q * 512 : sn + (q - 4) * 512);
          uint32_t r[16];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            r[q] = v[q].x;
            r[4 + q] = v[q].y;
            r[8 + q] = v[q].z;
            r[12 + q] = v[q].w;
          }
          tmem_st_32x32b_x16(col, r);
          uint32_t w[32];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            w[q] = v[4 + q].x;
            w[8 + q] = v[4 + q].y;
            w[16 + q] = v[4 + q].z;
            w[24 + q] = v[4 + q].w;
          }
          tmem_st_32x32b_x32(col + F4_SF_N, w);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(map_to_cta(&tail->sf_full[stage], first));
        if (++stage == F4_STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  } else if (kSplit && warp >= F4_FIRST_EPI) {
    // ------------------------------------------------------------ results of a shared tile
    const int quarter = warp & 3, part = (warp - F4_FIRST_EPI) >> 2;
    const TensorScales by = tensor_scales(args.alpha_a, args.alpha_b);
    const float scale = by.scale;
    const Fp4Tile t = fp4_tile(args, first_tile);
    // the whole sum within one limit, which receive_sums counts on: at most F4_MAX_SHARE stages
    const bool ok = __all_sync(0xffffffffu, pair_wait(&tail->acc_full, 0, abort_flag));
    tc_fence_after();
    const int rows = t.r_end - t.r0, slot = quarter * 32 + lane;
    const int f = t.f0 + static_cast<int>(rank) * 128 + slot;
    const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    // 2 columns at a time, every fourth stretch of 2 to a warp
    if (pair > 0) {
      // this CTA's sums [row][128 features] to the start of its ring (its MMAs are done), and from
      // there in one copy to the first pair's CTA; plain remote stores took 0.2 us a row
      float* mine = reinterpret_cast<float*>(smem) + slot;
      for (int c = part * 2; ok && c < rows; c += 8) {
        uint32_t v[2];
        tmem_ld_32x32b_x2(from + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (c + j < rows) mine[(c + j) * 128] = __uint_as_float(v[j]);
      }
      fence_proxy_async_smem();
      asm volatile("bar.sync 1, %0;" ::"n"(32 * F4_EPI_WARPS) : "memory");
      if (warp == F4_FIRST_EPI && lane == 0)
        send_sums(ok, map_to_cta(tail->sums + (pair - 1) * rows * 128, rank), smem, static_cast<uint32_t>(rows) * 512,
                  map_to_cta(&tail->sums_full, rank));
    } else if (receive_sums(ok, &tail->sums_full, abort_flag)) {
      for (int c = part * 2; c < rows; c += 8) {
        uint32_t v[2];
        tmem_ld_32x32b_x2(from + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (c + j >= rows || f >= args.n) continue;
          float sum = __uint_as_float(v[j]);
#pragma unroll
          for (int q = 0; q < F4_MAX_SPLIT - 1; ++q)
            if (q < args.split - 1) sum += tail->sums[(q * rows + c + j) * 128 + slot];
          sum *= by.first;
          const int64_t to = static_cast<int64_t>(t.r0 + c + j) * args.ldo + f;
          if constexpr (OUT == kTypeFp32)
            static_cast<float*>(args.out)[to] = sum * scale;
          else
            static_cast<uint16_t*>(args.out)[to] = static_cast<uint16_t>(pack_pair<OUT>(sum * scale, 0.0f));
        }
      }
    }
  } else if (warp >= F4_FIRST_EPI) {
    // ------------------------------------------------------------ results
    const int quarter = warp & 3, part = (warp - F4_FIRST_EPI) >> 2;  // 64 columns of a lane quarter
    const TensorScales by = tensor_scales(args.alpha_a, args.alpha_b);
    const float scale = by.scale;
    // two features of a row go as one 4-byte store where every row starts on 4 bytes
    const bool pairs =
        ((args.n | args.ldo) & 1) == 0 && (reinterpret_cast<uintptr_t>(args.out) & 3) == 0;
    uint32_t acc_phase = 0;
    for (int id = first_tile; id < total; id += tile_stride) {
      const Fp4Tile t = fp4_tile(args, id);
      if (!__all_sync(0xffffffffu, pair_wait(&tail->acc_full, acc_phase, abort_flag, kWaitLimitNs, progress))) break;
      acc_phase ^= 1;
      tc_fence_after();
      const int c0 = part * 64;
      uint32_t v[2][32];
      const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c0;
      if (c0 < t.n) tmem_ld_32x32b_x32(from, v[0]);
      if (c0 + 32 < t.n) tmem_ld_32x32b_x32(from + 32, v[1]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(map_to_cta(&tail->acc_empty, first));
      if (by.first != 1.0f) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 32; ++j) v[h][j] = __float_as_uint(__uint_as_float(v[h][j]) * by.first);
      }
      // a lane holds feature f of 32 consecutive rows, twice
      const int f = t.f0 + static_cast<int>(rank) * 128 + quarter * 32 + lane;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = t.r0 + c0 + h * 32;
        if (c0 + h * 32 >= t.n) break;
        if constexpr (OUT == kTypeFp32) {
          float* p = static_cast<float*>(args.out) + static_cast<int64_t>(row) * args.ldo + f;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (row + j < t.r_end && f < args.n) p[j * args.ldo] = __uint_as_float(v[h][j]) * scale;
        } else if (pairs) {
          // two rows of a lane's feature trade places with the neighbouring lane's, so that each
          // lane stores two features of one row; without comparisons where the tile is whole (at
          // K = 1536, where the results take as long as the sums, they were 15% of the product)
          const int odd = lane & 1;
          uint16_t* p = static_cast<uint16_t*>(args.out) + static_cast<int64_t>(row + odd) * args.ldo + (f - odd);
          if (row + 32 <= t.r_end && t.f0 + 256 <= args.n) {
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              *reinterpret_cast<uint32_t*>(p) = trade_pair<OUT>(v[h][j], v[h][j + 1], scale, odd);
              p += 2 * args.ldo;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const uint32_t w = trade_pair<OUT>(v[h][j], v[h][j + 1], scale, odd);
              if (row + j + odd < t.r_end && f < args.n) *reinterpret_cast<uint32_t*>(p) = w;
              p += 2 * args.ldo;
            }
          }
        } else {  // rows that may start on odd elements: one value at a time
          uint16_t* p = static_cast<uint16_t*>(args.out) + static_cast<int64_t>(row) * args.ldo + f;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const uint32_t w = pack_pair<OUT>(__uint_as_float(v[h][j]) * scale, 0.0f);
            if (row + j < t.r_end && f < args.n) p[j * args.ldo] = static_cast<uint16_t>(w);
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the other may still signal or read it
  tc_fence_after();
  if (threadIdx.x == 0 && tail->abort_flag) atomicOr(&g_fp4_err, kErrTimeoutMma);
  if (warp == 3) tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------------------ host
bool make_bytes_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t pitch, uint32_t box_cols,
                    uint32_t box_rows, bool swizzle) {
  auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
  if (!enc) return false;
  cuuint64_t dim[2] = {cols, rows};
  cuuint64_t stride[1] = {pitch};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dim, stride, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FORMAT, int OUT, bool kSplit>
cudaError_t launch_fp4_as(const Fp4Args& a, const Fp4Maps& maps, unsigned grid, unsigned cluster, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(gemm_fp4_kernel<FORMAT, OUT, kSplit>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kFp4Smem));
  if (e != cudaSuccess) return e;
  return launch_pdl_clusters(gemm_fp4_kernel<FORMAT, OUT, kSplit>, grid, cluster, F4_THREADS, kFp4Smem, s, a, maps);
}

template <int FORMAT, int OUT>
cudaError_t launch_fp4(Fp4Args a, const Fp4Maps& maps, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(a.blocks) * ((a.n + F4_TILE - 1) / F4_TILE);
  // As many pairs to a tile of one row block as leave no SM idle, as far as the first can receive
  // their sums, in clusters of up to eight CTAs, and each with a ring's worth of K steps at least:
  // the exchange takes as long as those.  A longer share than F4_MAX_SHARE is not waited for in one
  // piece: such a tile is left to one pair.
  const int64_t steps = (a.k + F4_BK - 1) / F4_BK;
  const int64_t fit = a.blocks == 1 ? 1 + F4_SUM_ROWS / a.m : 1;
  a.split = static_cast<int>(std::min({int64_t{F4_MAX_SPLIT}, sms / 2 / tiles, steps / F4_STAGES, fit}));
  if (a.split > 1 && (steps + a.split - 1) / a.split <= F4_MAX_SHARE)
    return launch_fp4_as<FORMAT, OUT, true>(a, maps, static_cast<unsigned>(tiles * 2 * a.split),
                                            static_cast<unsigned>(2 * a.split), s);
  a.split = 1;
  return launch_fp4_as<FORMAT, OUT, false>(a, maps, static_cast<unsigned>(2 * std::min<int64_t>(sms / 2, tiles)), 2, s);
}

template <int FORMAT>
cudaError_t launch_format(int out_type, const Fp4Args& a, const Fp4Maps& maps, cudaStream_t s) {
  if (out_type == kTypeBf16) return launch_fp4<FORMAT, kTypeBf16>(a, maps, s);
  if (out_type == kTypeFp16) return launch_fp4<FORMAT, kTypeFp16>(a, maps, s);
  return launch_fp4<FORMAT, kTypeFp32>(a, maps, s);
}

bool on(const void* p, uintptr_t a) { return p && aligned_to(p, a); }

}  // namespace

cudaError_t gemm_fp4_error_word(uint32_t** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_fp4_err);
}

}  // namespace beam

using namespace beam;

extern "C" beam_moe_status beam_moe_gemm_fp4(int32_t format, const uint8_t* a_codes, int64_t lda, const uint8_t* a_sf,
                                             int64_t lda_sf, const float* alpha_a, const uint8_t* b_codes, int64_t ldb,
                                             const uint8_t* b_sf, int64_t ldb_sf, const float* alpha_b, int32_t m,
                                             int32_t n, int32_t k, void* out, int32_t out_type, int64_t ldo,
                                             void* stream) {
  if (m < 0 || n < 0 || k < 1 || (format != BEAM_MOE_FP4_MX && format != BEAM_MOE_FP4_NV)) return BEAM_MOE_ERR_INVALID_ARG;
  if (out_type != BEAM_MOE_BF16 && out_type != BEAM_MOE_FP16 && out_type != BEAM_MOE_FP32) return BEAM_MOE_ERR_INVALID_ARG;
  if (k % 32 != 0 || m > 0x7fff0000 || n > 0x7fff0000 || k > 0x7fff0000) return BEAM_MOE_ERR_UNSUPPORTED;
  if ((static_cast<int64_t>(m) + 255) / 256 * ((static_cast<int64_t>(n) + 255) / 256) > (1 << 30))
    return BEAM_MOE_ERR_UNSUPPORTED;
  if (m == 0 || n == 0) return BEAM_MOE_OK;
  const int64_t scales = k / (format == BEAM_MOE_FP4_MX ? 32 : 16);
  if (!on(a_codes, 16) || !on(b_codes, 16) || !on(a_sf, 16) || !on(b_sf, 16) ||
      !on(out, out_type == BEAM_MOE_FP32 ? 4 : 2))
    return BEAM_MOE_ERR_INVALID_ARG;
  if ((alpha_a && !on(alpha_a, 4)) || (alpha_b && !on(alpha_b, 4))) return BEAM_MOE_ERR_INVALID_ARG;
  if (lda < k / 2 || ldb < k / 2 || lda % 16 != 0 || ldb % 16 != 0 || lda_sf < scales || ldb_sf < scales ||
      lda_sf % 16 != 0 || ldb_sf % 16 != 0 || ldo < n)
    return BEAM_MOE_ERR_INVALID_ARG;
  const bool mx = format == BEAM_MOE_FP4_MX;
  const int64_t size = out_type == BEAM_MOE_FP32 ? 4 : 2;
  if (overlaps_any({out, m, n * size, ldo * size},
                   {{a_codes, m, k / 2, lda}, {a_sf, m, scales, lda_sf}, {b_codes, n, k / 2, ldb},
                    {b_sf, n, scales, ldb_sf}, {mx ? nullptr : alpha_a, 1, 4, 4}, {mx ? nullptr : alpha_b, 1, 4, 4}}))
    return BEAM_MOE_ERR_INVALID_ARG;
  const int blocks = (m + F4_TILE - 1) / F4_TILE;
  const int height = ((m + blocks - 1) / blocks + 31) / 32 * 32;
  Fp4Maps maps;
  if (!make_bytes_map(&maps.m_codes, b_codes, k / 2, n, ldb, 128, 128, true) ||
      !make_bytes_map(&maps.n_codes, a_codes, k / 2, m, lda, 128, height / 2, true) ||
      !make_bytes_map(&maps.m_sf, b_sf, scales, n, ldb_sf, 16, 128, false) ||
      !make_bytes_map(&maps.n_sf, a_sf, scales, m, lda_sf, 16, height, false))
    return BEAM_MOE_ERR_UNSUPPORTED;  // strides that a tensor map cannot hold
  // MXFP4 has no tensor scale
  const Fp4Args args{m, n, k, blocks, height, 1, mx ? nullptr : alpha_a, mx ? nullptr : alpha_b, out, ldo};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = mx ? launch_format<BEAM_MOE_FP4_MX>(out_type, args, maps, s)
                           : launch_format<BEAM_MOE_FP4_NV>(out_type, args, maps, s);
  return launch_status(e);
}
