// Matrix products grouped by expert with ragged sizes, for 16-bit experts (BF16 or FP16): rows
// sorted by expert, offsets[e] .. offsets[e + 1] the rows of expert e,
//   forward  y[r][n]     = sum_k x[r][k] w[e][n][k]
//   dgrad    dx[r][k]    = sum_n dy[r][n] w[e][n][k]
//   wgrad    dw[e][n][k] = sum over the rows r of e of dy[r][n] x[r][k]
// with FP32 accumulation in TMEM and one rounding of the result.  One persistent kernel,
// template MODE, on tcgen05.mma.kind::f16 over CTA pairs (256 x 256 output tiles).
//
// Which operand is which.  The tensor core's M is fixed (256 over the pair) and its N may be
// any multiple of 32: the ragged dimension, the rows of an expert, is therefore N, and the
// features are M.  An expert with 40 rows costs an N of 64 instead of a padded tile of 256, and
// a decoding step (one row for most experts) an N of 32, so that the kernel streams weights.
//             A operand (M)                  B operand (N)               reduction
//   forward   w[e], K-major: features n      x, K-major: rows            k
//   dgrad     w[e], M-major: features k      dy, K-major: rows           n
//   wgrad     dy, M-major: features n        x, N-major: features k      rows of e
// "M-major" operands lie in memory with the M dimension contiguous; TMA brings 64 values x 64
// reduction steps per chunk and the tensor core transposes (matrix descriptor and instruction
// descriptor say so), so that dgrad and wgrad need no transposed copy of weights or rows.
//
// Ragged edges.  Rows past an expert's last one are loaded with it (they belong to the next
// expert, or TMA fills zeros past the tensor) and only feed accumulator columns that are never
// stored.  In wgrad the rows are the reduction: a stage that holds rows past the last one gets
// them zeroed in shared memory, in BOTH operands (0 * inf would be NaN), by a warp that does
// nothing else, before the MMA sees it.
//
// A CTA (384 threads): warp 0 issues the TMA loads (6 stages of 32 KB: 64 reduction steps of
// this CTA's 128 M rows and of its half of the N rows), warp 1 of the leading CTA the MMAs,
// warp 2 zeroes the ragged stages of wgrad, warp 3 owns TMEM, warps 4..11 store the results.
// Two accumulators of 256 columns: a tile is stored while the next one is multiplied.
// Tiles are dealt out round robin; the order keeps the tiles that run together on the same
// weights (forward, dgrad) or the same expert (wgrad), whose operands L2 then holds.
//
// What bounds it.  A stage of an n-row tile is 2 n cycles of MMAs against about 256 + n for its
// operands on their way through L2 and shared memory: they meet at 256 rows, where the tensor pipe
// is active 89% of the cycles and the power limit sets the clock.  16384 x 5120 x 5120 BF16, from idle
// and in a loop of a second: one group 578 and 670 us (cuBLAS 563 and 644), 32 experts of 512 rows
// each 652 and 777; uneven experts lose to tiles of fewer rows (713 and 846).  With a row or a few for
// each expert it streams weights: 64 rows over 256 experts of 1536 x 5120 in 146 to 154 us, 5.8 to
// 6.1 TB/s.  A tile's sum is never divided: a product of few tiles leaves most pairs idle (gradient of
// 4 experts of 256 x 256 over 32768 rows: 41 us on 4 of 74 pairs).
//
// The work list comes from the offsets, which only the device knows: every CTA scans them at
// its start (at most 1024 experts).  They are read as their running maximum, clamped to
// [0, rows], so no offsets can make the kernel leave its buffers.
#include <cudaTypedefs.h>

#include <algorithm>

#include <cuda_fp16.h>

#include "../../include/beam_moe.h"
#include "cta_pair.cuh"
#include "internal.h"
#include "overlap.h"

namespace beam {

namespace {

__device__ uint32_t g_grouped_err;  // error bits of this device's grouped products

constexpr int kFwd = 0, kDgrad = 1, kWgrad = 2;

constexpr int GG_BK = 64;                        // reduction steps of a stage: one 128-byte line of 16-bit values
constexpr int GG_STAGES = 6;
constexpr int GG_OPERAND = 128 * GG_BK * 2;      // 16 KB: 128 rows (or columns) of one operand
constexpr int GG_STAGE = 2 * GG_OPERAND;
constexpr int GG_CHUNK = 64 * GG_BK * 2;         // 8 KB: 64 contiguous values x 64 reduction steps
constexpr int GG_BOX_ROWS = 32;                  // rows of one load of a K-major B operand
constexpr int GG_TILE = 256;
constexpr int GG_PANEL = 8;                      // row blocks that share an expert's weights in turn
constexpr int GG_EPI_WARPS = 8;
constexpr int GG_FIRST_EPI = 4;
constexpr int GG_THREADS = 32 * (GG_FIRST_EPI + GG_EPI_WARPS);
constexpr int GG_MAX_GROUPS = 1024;

struct GroupedArgs {
  const int32_t* offsets;
  int groups;
  int rows;       // rows of x / dy
  int m;          // features on the tensor core's M: n (forward, wgrad) or k (dgrad)
  int kdim;       // reduction length (forward, dgrad)
  int ncols;      // wgrad: k
  void* out;
  int64_t ldo;    // forward, dgrad: elements between rows of out
  int bf16;       // operand type
};

struct __align__(16) GroupedTail {
  // results on their way out: wgrad 32 rows x 64 bytes of each storing warp, else 32 rows x 128
  // features of each four
  uint8_t turn[GG_EPI_WARPS * 2048];
  uint64_t full[GG_STAGES];       // leader: both CTAs' halves have landed
  uint64_t empty[GG_STAGES];
  uint64_t landed[GG_STAGES];     // wgrad: this CTA's half of a ragged stage has landed
  uint64_t acc_full[2];
  uint64_t acc_empty[2];          // leader
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  uint32_t progress;              // stages loaded
  int total_tiles;
  int begin[GG_MAX_GROUPS + 1];   // clamped offsets
  int first[GG_MAX_GROUPS + 1];   // first tile of each group
};

constexpr size_t kGroupedSmem = static_cast<size_t>(GG_STAGES) * GG_STAGE + sizeof(GroupedTail) + 1024;
static_assert(kGroupedSmem <= 227 * 1024, "shared memory of one CTA");

// One output tile: M features [m0, m0 + 256) and N columns [n0, n0 + n), n a multiple of 32.
struct GroupedTile {
  int group, m0, n0, n;
  int n_end;   // forward, dgrad: rows from n0 up to here are the tile's
  int steps;   // stages of the reduction
};

template <int MODE>
__device__ __forceinline__ GroupedTile grouped_tile(const GroupedArgs& a, const GroupedTail* s, int id) {
  GroupedTile t;
  const int mt = (a.m + GG_TILE - 1) / GG_TILE;
  if (MODE == kWgrad) {
    const int nt = (a.ncols + GG_TILE - 1) / GG_TILE;
    t.group = id / (mt * nt);
    const int rest = id - t.group * mt * nt;
    t.m0 = rest / nt * GG_TILE;
    t.n0 = rest % nt * GG_TILE;
    t.n = min(GG_TILE, (a.ncols - t.n0 + 31) & ~31);
    t.n_end = a.ncols;
    t.steps = (s->begin[t.group + 1] - s->begin[t.group] + GG_BK - 1) / GG_BK;
    return t;
  }
  int lo = 0, hi = a.groups - 1;  // the last group whose first tile is <= id
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s->first[mid] <= id) lo = mid; else hi = mid - 1;
  }
  t.group = lo;
  const int begin = s->begin[lo], rows = s->begin[lo + 1] - begin;
  const int blocks = (rows + GG_TILE - 1) / GG_TILE;
  int rest = id - s->first[lo];
  // panels of row blocks; in a panel the row blocks of one feature tile come one after another
  const int panel = rest / (GG_PANEL * mt);
  rest -= panel * GG_PANEL * mt;
  const int wide = min(GG_PANEL, blocks - panel * GG_PANEL);
  t.m0 = rest / wide * GG_TILE;
  const int block = panel * GG_PANEL + rest % wide;
  // equal blocks rather than full ones and a rest: the last block's MMAs would run at a small N
  const int height = ((rows + blocks - 1) / blocks + 31) & ~31;
  t.n0 = begin + block * height;
  t.n_end = min(begin + rows, t.n0 + height);
  t.n = max(32, (t.n_end - t.n0 + 31) & ~31);
  t.steps = (a.kdim + GG_BK - 1) / GG_BK;
  return t;
}

template <int MODE, int OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GG_THREADS, 1)
    grouped_gemm_kernel(const GroupedArgs args, const __grid_constant__ CUtensorMap map_a,
                        const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_b128) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  GroupedTail* tail = reinterpret_cast<GroupedTail*>(smem + GG_STAGES * GG_STAGE);
  volatile int* abort_flag = &tail->abort_flag;
  volatile uint32_t* progress = &tail->progress;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_cta_rank();

  if (threadIdx.x == 0) {
    prefetch_tmap(&map_a);
    prefetch_tmap(&map_b);
    for (int i = 0; i < GG_STAGES; ++i) {
      mbar_init(&tail->full[i], 2);
      mbar_init(&tail->empty[i], 1);
      mbar_init(&tail->landed[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tail->acc_full[i], 1);
      mbar_init(&tail->acc_empty[i], 2 * GG_EPI_WARPS);
    }
    mbar_init(&tail->drain, 1);
    tail->abort_flag = 0;
    tail->progress = 0;
    fence_mbar_init();
  }
  if (warp == 3) {
    tmem_alloc_pair(&tail->tmem_base, 512);
    tmem_relinquish_pair();
  }
  pdl_wait();
  pdl_trigger();
  // The groups' borders and first tiles.
  for (int e = threadIdx.x; e <= args.groups; e += GG_THREADS)
    tail->begin[e] = min(max(__ldcg(args.offsets + e), 0), args.rows);
  __syncthreads();
  if (warp == 0) {
    const int mt = (args.m + GG_TILE - 1) / GG_TILE;
    int top = 0, sum = 0;
    int carry = 0;  // border of the group before
    for (int e0 = 0; e0 <= args.groups; e0 += 32) {
      const int e = e0 + lane;
      int v = e <= args.groups ? tail->begin[e] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = max(v, u);
      }
      v = max(v, top);
      top = __shfl_sync(0xffffffffu, v, 31);
      int prev = __shfl_up_sync(0xffffffffu, v, 1);
      if (lane == 0) prev = e0 == 0 ? v : carry;
      carry = top;
      // tiles of group e - 1, summed up to and with it: the first tile of group e
      int c = ((v - prev + GG_TILE - 1) / GG_TILE) * mt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += u;
      }
      c += sum;
      sum = __shfl_sync(0xffffffffu, c, 31);
      if (e <= args.groups) {
        tail->begin[e] = v;
        tail->first[e] = c;
      }
    }
    if (lane == 0)
      tail->total_tiles = MODE == kWgrad ? args.groups * mt * ((args.ncols + GG_TILE - 1) / GG_TILE) : sum;
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers are set before anyone arrives at them
  tc_fence_after();
  const uint32_t tmem = tail->tmem_base;
  const int total = tail->total_tiles;
  const int first_tile = blockIdx.x >> 1, tile_stride = gridDim.x >> 1;

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    int stage = 0;
    uint32_t phase = 0, loaded = 0;
    bool ok = true;
    for (int id = first_tile; id < total && ok; id += tile_stride) {
      const GroupedTile t = grouped_tile<MODE>(args, tail, id);
      const int half = t.n >> 1;
      const int b_boxes = MODE == kWgrad ? (half + 63) / 64 : (half + GG_BOX_ROWS - 1) / GG_BOX_ROWS;
      const uint32_t bytes = GG_OPERAND + static_cast<uint32_t>(b_boxes) * (MODE == kWgrad ? GG_CHUNK : GG_BOX_ROWS * 128);
      const int m0 = t.m0 + static_cast<int>(rank) * 128, n0 = t.n0 + static_cast<int>(rank) * half;
      const int begin = MODE == kWgrad ? tail->begin[t.group] : 0;
      const int length = MODE == kWgrad ? tail->begin[t.group + 1] - begin : 0;
      for (int i = 0; i < t.steps; ++i) {
        ok = __all_sync(0xffffffffu, pair_wait(&tail->empty[stage], phase ^ 1, abort_flag));
        if (!ok) break;
        uint8_t* sa = smem + stage * GG_STAGE;
        uint8_t* sb = sa + GG_OPERAND;
        const int step = i * GG_BK;
        // a ragged stage lands on this CTA's own barrier; warp 2 hands it on
        const bool ragged = MODE == kWgrad && i == t.steps - 1 && (length & 15) != 0;
        ++loaded;
        if (elect_one()) {
          *progress = loaded;
          const uint32_t bar = ragged ? map_to_cta(&tail->landed[stage], rank) : map_to_cta(&tail->full[stage], 0);
          mbar_arrive_expect_tx_relaxed_at(bar, bytes);
          if (MODE == kFwd) {
            tma_load_3d_pair(sa, &map_a, bar, step, m0, t.group);
          } else if (MODE == kDgrad) {
            tma_load_3d_pair(sa, &map_a, bar, m0, step, t.group);
            tma_load_3d_pair(sa + GG_CHUNK, &map_a, bar, m0 + 64, step, t.group);
          } else {
            tma_load_2d_pair(sa, &map_a, bar, m0, begin + step);
            tma_load_2d_pair(sa + GG_CHUNK, &map_a, bar, m0 + 64, begin + step);
          }
          if (MODE == kWgrad) {
            tma_load_2d_pair(sb, &map_b, bar, n0, begin + step);
            if (b_boxes == 2) tma_load_2d_pair(sb + GG_CHUNK, &map_b, bar, n0 + 64, begin + step);
          } else if (half == 128) {
            tma_load_2d_pair(sb, &map_b128, bar, step, n0);
          } else {
            for (int b = 0; b < b_boxes; ++b)
              tma_load_2d_pair(sb + b * GG_BOX_ROWS * 128, &map_b, bar, step, n0 + b * GG_BOX_ROWS);
          }
        }
        __syncwarp();
        if (++stage == GG_STAGES) {
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
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, ready = false;
      const uint32_t leader = elect_one() ? 1u : 0u;
      const uint32_t type = args.bf16 ? 1u : 0u;
      // FP32 accumulator, operand types, M- and N-major operands, M = 256
      const uint32_t idesc0 = (1u << 4) | (type << 7) | (type << 10) | ((MODE != kFwd ? 1u : 0u) << 15) |
                              ((MODE == kWgrad ? 1u : 0u) << 16) | ((GG_TILE >> 4) << 24);
      // Descriptors of stage 0; their low words hold the address in units of 16 bytes.  16
      // reduction steps further: 32 bytes of each line, or 16 lines of each chunk.
      constexpr uint32_t kStepA = MODE == kFwd ? 32 / 16 : 2048 / 16, kStepB = MODE == kWgrad ? 2048 / 16 : 32 / 16;
      const uint32_t base = smem_u32(smem);
      const uint64_t da0 = MODE == kFwd ? sdesc_k_sw128(base) : sdesc_mn_sw128(base, GG_CHUNK);
      const uint64_t db0 =
          MODE == kWgrad ? sdesc_mn_sw128(base + GG_OPERAND, GG_CHUNK) : sdesc_k_sw128(base + GG_OPERAND);
      for (int id = first_tile; id < total && ok; id += tile_stride) {
        const GroupedTile t = grouped_tile<MODE>(args, tail, id);
        if (t.steps == 0) continue;
        ok = __all_sync(0xffffffffu, pair_wait(&tail->acc_empty[acc], acc_phase ^ 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const uint32_t idesc = idesc0 | (static_cast<uint32_t>(t.n >> 3) << 17);
        const uint32_t d = tmem + acc * GG_TILE;
        const int length = MODE == kWgrad ? tail->begin[t.group + 1] - tail->begin[t.group] : args.kdim;
        for (int i = 0; i < t.steps; ++i) {
          if (!ready) {
            ok = __all_sync(0xffffffffu, pair_wait(&tail->full[stage], phase, abort_flag));
            if (!ok) break;
          }
          tc_fence_after();
          // look at the next stage's barrier while this stage's MMAs go out
          const int next = stage + 1 == GG_STAGES ? 0 : stage + 1;
          const uint32_t next_phase = phase ^ (next == 0 ? 1u : 0u);
          const bool next_ready = mbar_test(&tail->full[next], next_phase);
          const uint64_t da = da0 + static_cast<uint64_t>(stage * (GG_STAGE / 16));
          const uint64_t db = db0 + static_cast<uint64_t>(stage * (GG_STAGE / 16));
          const int left = length - i * GG_BK;
#pragma unroll
          for (int j = 0; j < GG_BK / 16; ++j)
            if (j * 16 < left) tc_mma_f16_pair(d, da + j * kStepA, db + j * kStepB, idesc, (i | j) != 0 ? 1u : 0u, leader);
          tc_commit_pair(&tail->empty[stage], leader);
          stage = next;
          phase = next_phase;
          ready = __all_sync(0xffffffffu, next_ready);
        }
        if (!ok) break;
        tc_commit_pair(&tail->acc_full[acc], leader);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      if (!ok) {  // nothing may read shared memory or write TMEM after the CTAs are gone
        tc_commit_pair(&tail->drain, leader);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&tail->drain, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ ragged stages of wgrad
    if (MODE == kWgrad) {
      int stage = 0;
      uint32_t parity = 0;  // one bit per stage
      bool ok = true;
      for (int id = first_tile; id < total && ok; id += tile_stride) {
        const GroupedTile t = grouped_tile<MODE>(args, tail, id);
        if (t.steps == 0) continue;
        const int last = (stage + t.steps - 1) % GG_STAGES;
        stage = (stage + t.steps) % GG_STAGES;
        const int rows = tail->begin[t.group + 1] - tail->begin[t.group] - (t.steps - 1) * GG_BK;
        if ((rows & 15) == 0) continue;
        ok = pair_wait(&tail->landed[last], (parity >> last) & 1u, abort_flag, kWaitLimitNs, progress);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        parity ^= 1u << last;
        uint8_t* base = smem + last * GG_STAGE;
        const int chunks = 2 + ((t.n >> 1) + 63) / 64;  // A's two, then B's
        const int zero_rows = ((rows + 15) & ~15) - rows;
        for (int q = lane; q < chunks * zero_rows * 8; q += 32) {
          const int c = q / (zero_rows * 8), r = q / 8 % zero_rows, p = q & 7;
          *reinterpret_cast<uint4*>(base + c * GG_CHUNK + (rows + r) * 128 + p * 16) = make_uint4(0, 0, 0, 0);
        }
        // The zeros are in this SM's shared memory, for the tensor core that reads it there, once
        // the proxy fence has passed: the arrival that follows needs to carry nothing else.  (With a
        // release at cluster scope, in turn: 46.4 against 44.1 us for 3001 rows of 48 experts, 520 x
        // 1000, FP16; no difference for 512 rows an expert.)
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(map_to_cta(&tail->full[last], 0));
      }
    }
  } else if (warp >= GG_FIRST_EPI) {
    // ------------------------------------------------------------ results
    const int w = warp - GG_FIRST_EPI;
    const int quarter = warp & 3;          // the warp's lanes of TMEM
    const int side = w >> 2;               // and its half of the columns
    int acc = 0;
    uint32_t acc_phase = 0;
    // Once a wait gave up, the tiles are gone through without waits and without stores to the end:
    // the warps that share a named barrier meet at it all the same.
    bool ok = true;
    for (int id = first_tile; id < total; id += tile_stride) {
      const GroupedTile t = grouped_tile<MODE>(args, tail, id);
      const bool any = t.steps > 0;
      if (any) {
        ok = ok && __all_sync(0xffffffffu, pair_wait(&tail->acc_full[acc], acc_phase, abort_flag, kWaitLimitNs, progress));
        tc_fence_after();
      }
      const int m = t.m0 + static_cast<int>(rank) * 128 + quarter * 32 + lane;
      for (int c = side * 32; c < t.n; c += 64) {
        uint32_t v[32];
        if (any) {
          tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + acc * GG_TILE + c, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0;
        }
        if constexpr (MODE == kWgrad) {
          // A lane holds 32 consecutive values of dw's row m.  Through shared memory, so that four
          // neighbouring lanes store 64 bytes of one row and an instruction touches 8 rows: stored
          // from the lanes that hold them (32 rows an instruction), the results of 512 rows took
          // longer than their multiplication (290 against 191 us with no stores at all).
          constexpr int kBytes = OUT == kTypeFp32 ? 4 : 2;
          constexpr int kCols = 64 / kBytes;  // columns of one pass: 64 bytes of each row
          uint8_t* tile = tail->turn + w * 2048;
          const int sub = lane >> 2, part = lane & 3;
#pragma unroll
          for (int h = 0; h < 32 / kCols; ++h) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // 16-byte part j of row `lane`, turned so that no banks collide
              uint4 q;
              if constexpr (OUT == kTypeFp32) {
                const uint32_t* f = v + h * kCols + 4 * j;
                q = make_uint4(f[0], f[1], f[2], f[3]);
              } else {
                const uint32_t* f = v + 8 * j;
                q.x = pack_pair<OUT>(__uint_as_float(f[0]), __uint_as_float(f[1]));
                q.y = pack_pair<OUT>(__uint_as_float(f[2]), __uint_as_float(f[3]));
                q.z = pack_pair<OUT>(__uint_as_float(f[4]), __uint_as_float(f[5]));
                q.w = pack_pair<OUT>(__uint_as_float(f[6]), __uint_as_float(f[7]));
              }
              *reinterpret_cast<uint4*>(tile + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = q;
            }
            __syncwarp();
            const int col = t.n0 + c + h * kCols + part * (16 / kBytes);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 8 * i + sub, row = m - lane + r;
              const uint4 q = *reinterpret_cast<const uint4*>(tile + r * 64 + ((part ^ ((r >> 1) & 3)) << 4));
              if (ok && row < args.m && col < args.ncols)
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(args.out) +
                                          ((static_cast<int64_t>(t.group) * args.m + row) * args.ncols + col) * kBytes) = q;
            }
          }
        } else {
          // a lane holds feature m of 32 consecutive rows
          const int row = t.n0 + c;
          if constexpr (OUT == kTypeFp32) {
            float* p = static_cast<float*>(args.out) + static_cast<int64_t>(row) * args.ldo + m;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (ok && row + j < t.n_end && m < args.m) p[j * args.ldo] = __uint_as_float(v[j]);
          } else {
            store_turned<OUT>(v, tail->turn + side * 8192, 1 + side, quarter, lane,
                              static_cast<uint16_t*>(args.out), args.ldo, row, ok ? t.n_end : row,
                              t.m0 + static_cast<int>(rank) * 128, args.m);
          }
        }
      }
      if (any) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(map_to_cta(&tail->acc_empty[acc], 0));
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the other may still signal or read it
  tc_fence_after();
  if (threadIdx.x == 0 && tail->abort_flag) atomicOr(&g_grouped_err, kErrTimeoutMma);
  if (warp == 3) tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------------------ host
bool make_map(CUtensorMap* m, int bf16, const void* base, int dims, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1,
              uint64_t s2, uint32_t b0, uint32_t b1) {
  auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
  if (!enc) return false;
  cuuint64_t dim[3] = {d0, d1, d2};
  cuuint64_t stride[2] = {s1, s2};
  cuuint32_t box[3] = {b0, b1, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dims,
             const_cast<void*>(base), dim, stride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int OUT>
cudaError_t launch_mode(const GroupedArgs& a, const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mb2, int64_t most_tiles,
                        cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(grouped_gemm_kernel<MODE, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kGroupedSmem));
  if (e != cudaSuccess) return e;
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(sms / 2, most_tiles));
  return launch_pdl(grouped_gemm_kernel<MODE, OUT>, dim3(static_cast<unsigned>(2 * pairs)), dim3(GG_THREADS),
                    kGroupedSmem, s, a, ma, mb, mb2);
}

template <int MODE>
cudaError_t launch_out(int out_type, const GroupedArgs& a, const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mb2,
                       int64_t most_tiles, cudaStream_t s) {
  if (out_type == kTypeBf16) return launch_mode<MODE, kTypeBf16>(a, ma, mb, mb2, most_tiles, s);
  if (out_type == kTypeFp16) return launch_mode<MODE, kTypeFp16>(a, ma, mb, mb2, most_tiles, s);
  return launch_mode<MODE, kTypeFp32>(a, ma, mb, mb2, most_tiles, s);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

int64_t grouped_gemm_most_tiles(int mode, int64_t rows, int64_t groups, int64_t n, int64_t k) {
  if (mode == kWgrad) return groups * ceil_div(n, GG_TILE) * ceil_div(k, GG_TILE);
  return (rows / GG_TILE + std::min(groups, rows)) * ceil_div(mode == kDgrad ? k : n, GG_TILE);
}

cudaError_t launch_grouped_gemm(int mode, const void* rows_a, int64_t ld_a, const void* rows_b, int64_t ld_b,
                                const void* w, const int32_t* offsets, int64_t rows, int groups, int n, int k,
                                int in_type, void* out, int64_t ldo, int out_type, cudaStream_t s) {
  const int bf16 = in_type == kTypeBf16;
  CUtensorMap ma, mb, mb2;
  bool ok;
  GroupedArgs a{offsets, groups, static_cast<int>(rows), mode == kDgrad ? k : n, mode == kDgrad ? n : k, k, out, ldo,
                bf16};
  const uint64_t row_w = static_cast<uint64_t>(k) * 2, mat_w = row_w * static_cast<uint64_t>(n);
  if (mode == kWgrad) {
    ok = make_map(&ma, bf16, rows_b, 2, n, rows, 1, ld_b * 2, 0, 64, 64) &&
         make_map(&mb, bf16, rows_a, 2, k, rows, 1, ld_a * 2, 0, 64, 64);
    mb2 = mb;
  } else {
    ok = make_map(&ma, bf16, w, 3, k, n, groups, row_w, mat_w, 64, mode == kFwd ? 128 : 64) &&
         make_map(&mb, bf16, rows_a, 2, mode == kFwd ? k : n, rows, 1, ld_a * 2, 0, 64, GG_BOX_ROWS) &&
         make_map(&mb2, bf16, rows_a, 2, mode == kFwd ? k : n, rows, 1, ld_a * 2, 0, 64, 128);
  }
  if (!ok) return cudaErrorNotSupported;  // strides that a tensor map cannot hold
  const int64_t tiles = grouped_gemm_most_tiles(mode, rows, groups, n, k);
  if (mode == kFwd) return launch_out<kFwd>(out_type, a, ma, mb, mb2, tiles, s);
  if (mode == kDgrad) return launch_out<kDgrad>(out_type, a, ma, mb, mb2, tiles, s);
  return launch_out<kWgrad>(out_type, a, ma, mb, mb2, tiles, s);
}

cudaError_t grouped_gemm_error_word(uint32_t** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_grouped_err);
}

}  // namespace beam

using namespace beam;

namespace {

// The checks that the three products share.
beam_moe_status check_grouped(int32_t rows, int32_t groups, int32_t n, int32_t k, int32_t type, int32_t out_type) {
  if (rows < 0 || groups < 1 || n < 1 || k < 1) return BEAM_MOE_ERR_INVALID_ARG;
  if ((type != BEAM_MOE_BF16 && type != BEAM_MOE_FP16) || (out_type != type && out_type != BEAM_MOE_FP32))
    return BEAM_MOE_ERR_INVALID_ARG;
  // 2^30: features and tile numbers stay in 32 bits with a tile or a grid to spare
  if (n % 8 != 0 || k % 8 != 0 || n > (1 << 30) || k > (1 << 30) || groups > GG_MAX_GROUPS || rows > 0x7fff0000)
    return BEAM_MOE_ERR_UNSUPPORTED;
  return BEAM_MOE_OK;
}

// A [rows][cols] operand whose rows are ld elements apart.
bool good_rows(const void* p, int64_t ld, int32_t cols) { return p && aligned_to(p, 16) && ld >= cols && ld % 8 == 0; }

Span rows_span(const void* p, int32_t rows, int32_t cols, int64_t ld, int32_t type) {
  const int64_t size = type == BEAM_MOE_FP32 ? 4 : 2;
  return {p, rows, cols * size, ld * size};
}
Span weights_span(const void* p, int32_t groups, int32_t n, int32_t k, int32_t type) {
  const int64_t row = static_cast<int64_t>(k) * (type == BEAM_MOE_FP32 ? 4 : 2);
  return {p, static_cast<int64_t>(groups) * n, row, row};
}
Span offsets_span(const int32_t* p, int32_t groups) { return {p, groups + 1, 4, 4}; }

}  // namespace

extern "C" {

beam_moe_status beam_moe_grouped_gemm(const void* x, int64_t ldx, const void* w, const int32_t* offsets, int32_t rows,
                                      int32_t groups, int32_t n, int32_t k, int32_t type, void* y, int64_t ldy,
                                      int32_t out_type, void* stream) {
  const beam_moe_status st = check_grouped(rows, groups, n, k, type, out_type);
  if (st != BEAM_MOE_OK) return st;
  if (grouped_gemm_most_tiles(kFwd, rows, groups, n, k) > (1 << 30)) return BEAM_MOE_ERR_UNSUPPORTED;
  if (rows == 0) return BEAM_MOE_OK;
  if (!good_rows(x, ldx, k) || !good_rows(y, ldy, n) || !w || !aligned_to(w, 16) || !offsets ||
      !aligned_to(offsets, 4))
    return BEAM_MOE_ERR_INVALID_ARG;
  if (overlaps_any(rows_span(y, rows, n, ldy, out_type),
                   {rows_span(x, rows, k, ldx, type), weights_span(w, groups, n, k, type), offsets_span(offsets, groups)}))
    return BEAM_MOE_ERR_INVALID_ARG;
  return launch_status(launch_grouped_gemm(kFwd, x, ldx, nullptr, 0, w, offsets, rows, groups, n, k, type, y, ldy,
                                           out_type, static_cast<cudaStream_t>(stream)));
}

beam_moe_status beam_moe_grouped_gemm_dgrad(const void* dy, int64_t lddy, const void* w, const int32_t* offsets,
                                            int32_t rows, int32_t groups, int32_t n, int32_t k, int32_t type, void* dx,
                                            int64_t lddx, int32_t out_type, void* stream) {
  const beam_moe_status st = check_grouped(rows, groups, n, k, type, out_type);
  if (st != BEAM_MOE_OK) return st;
  if (grouped_gemm_most_tiles(kDgrad, rows, groups, n, k) > (1 << 30)) return BEAM_MOE_ERR_UNSUPPORTED;
  if (rows == 0) return BEAM_MOE_OK;
  if (!good_rows(dy, lddy, n) || !good_rows(dx, lddx, k) || !w || !aligned_to(w, 16) || !offsets ||
      !aligned_to(offsets, 4))
    return BEAM_MOE_ERR_INVALID_ARG;
  if (overlaps_any(rows_span(dx, rows, k, lddx, out_type),
                   {rows_span(dy, rows, n, lddy, type), weights_span(w, groups, n, k, type), offsets_span(offsets, groups)}))
    return BEAM_MOE_ERR_INVALID_ARG;
  return launch_status(launch_grouped_gemm(kDgrad, dy, lddy, nullptr, 0, w, offsets, rows, groups, n, k, type, dx,
                                           lddx, out_type, static_cast<cudaStream_t>(stream)));
}

beam_moe_status beam_moe_grouped_gemm_wgrad(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                            const int32_t* offsets, int32_t rows, int32_t groups, int32_t n, int32_t k,
                                            int32_t type, void* dw, int32_t out_type, void* stream) {
  const beam_moe_status st = check_grouped(rows, groups, n, k, type, out_type);
  if (st != BEAM_MOE_OK) return st;
  if (grouped_gemm_most_tiles(kWgrad, rows, groups, n, k) > (1 << 30)) return BEAM_MOE_ERR_UNSUPPORTED;
  if (!dw || !aligned_to(dw, 16)) return BEAM_MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0)  // no rows: every gradient is zero
    return launch_status(cudaMemsetAsync(
        dw, 0, static_cast<size_t>(groups) * n * static_cast<size_t>(k) * (out_type == BEAM_MOE_FP32 ? 4 : 2), s));
  if (!good_rows(dy, lddy, n) || !good_rows(x, ldx, k) || !offsets || !aligned_to(offsets, 4))
    return BEAM_MOE_ERR_INVALID_ARG;
  if (overlaps_any(weights_span(dw, groups, n, k, out_type),
                   {rows_span(dy, rows, n, lddy, type), rows_span(x, rows, k, ldx, type), offsets_span(offsets, groups)}))
    return BEAM_MOE_ERR_INVALID_ARG;
  return launch_status(launch_grouped_gemm(kWgrad, x, ldx, dy, lddy, nullptr, offsets, rows, groups, n, k, type, dw, k,
                                           out_type, s));
}

}  // extern "C"
