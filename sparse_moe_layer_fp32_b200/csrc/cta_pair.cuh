// Device helpers for kernels whose CTAs work in pairs (clusters of two): one tcgen05.mma of
// cta_group::2 multiplies operands that lie half in each CTA's shared memory, and leaves
// accumulator rows 0..127 in the TMEM of CTA 0 and rows 128..255 in that of CTA 1.  The
// barriers that both CTAs signal live in CTA 0 (the leader), which issues the MMAs.
//
// The loads below carry no multicast: each CTA fetches its own half.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace beam {

// launch_pdl in clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl_clusters(void (*kernel)(KArgs...), unsigned grid, unsigned cluster, unsigned threads,
                                       size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

__device__ __forceinline__ uint32_t cluster_cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
// The address, in the cluster's shared window, of CTA `rank`'s copy of a shared variable.
__device__ __forceinline__ uint32_t map_to_cta(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}

// Copies `bytes` (a multiple of 16) of this CTA's shared memory to another CTA of the cluster,
// completing on a barrier there (addresses from map_to_cta).
__device__ __forceinline__ void bulk_copy_to_cta(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(smem_u32(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// Counts `bytes` as received at a barrier of another CTA, for a copy that will not be made.
__device__ __forceinline__ void mbar_complete_tx_at(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Arrivals at a barrier of either CTA (address from map_to_cta).  Plain: releases this thread's
// accesses to its own CTA only, which is right where what it announces are finished TMEM accesses
// or shared memory behind a proxy fence, both used only by the own SM's tensor core.  The relaxed
// one announces TMA copies (their bytes order themselves).  A release at cluster scope waits for
// outstanding stores; taken for every stage of a ring it cost ~1200 cycles per stage.
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx_relaxed_at(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// Whether the phase has completed, without suspending the thread.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait: false, with *abort_flag set, once the wait ran past the limit or another role gave
// up.  The clock is first read after kQuietTries tries (each suspends the
// thread for a while): reading %globaltimer takes about a microsecond, which on every wait that
// did not succeed at once held a ring stage to ~800 cycles.
// A role that waits for more than a stage of the ring (a whole sum, which may rightly take longer
// than the limit) passes `progress`, a word of this CTA's shared memory that the loading warp
// changes with every stage: the limit then counts from its last change.
constexpr uint32_t kQuietTries = 256;
__device__ __forceinline__ bool pair_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          uint64_t limit_ns = kWaitLimitNs,
                                          const volatile uint32_t* progress = nullptr) {
  uint64_t t0 = 0;
  uint32_t seen = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (i % kQuietTries == 0) {
      if (*abort_flag) return false;
      const uint64_t t = globaltimer_ns();
      const uint32_t at = progress ? *progress : 0u;
      if (t0 == 0 || at != seen) {
        t0 = t;
        seen = at;
      }
      if (t - t0 > limit_ns) {
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// The sums of a tile that several pairs share, on their way to the CTA that adds them up.  A sender
// whose own sums did not come (!ok) counts them as received all the same; one thread calls.
__device__ __forceinline__ void send_sums(bool ok, uint32_t to, const void* from, uint32_t bytes, uint32_t bar) {
  if (ok)
    bulk_copy_to_cta(to, from, bytes, bar);
  else
    mbar_complete_tx_at(bar, bytes);
}
// Whether this CTA's own sums (ok) and every sender's have come; whole warps call.  No sender's copy
// may find this CTA gone.  A sender decides within one wait limit of its start, the CTAs of a
// cluster start together, and a role here gives up one limit after that at the earliest: whoever
// gives up holds this CTA for another limit, unless all that will come has come before.
__device__ __forceinline__ bool receive_sums(bool ok, uint64_t* bar, volatile int* abort_flag,
                                             uint64_t limit_ns = kWaitLimitNs) {
  if (ok && __all_sync(0xffffffffu, pair_wait(bar, 0, abort_flag, limit_ns))) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
  }
  __syncwarp();
  return false;
}

// Tiled TMA loads into this CTA, completing on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                                 int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y,
                                                 int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, "
      "%4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// TMEM of both CTAs: one warp of each CTA makes the call.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* smem_dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_dst)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Arrives once on `bar` of both CTAs of the pair (`first` the cluster rank of its leading CTA) when
// every MMA issued before (by the lane that the converged warp elects, always the same one) has
// completed.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar, uint32_t leader, uint32_t first = 0) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3u << first)), "r"(leader)
      : "memory");
}
// One lane of a converged warp.  The roles that issue TMA copies and MMAs run as whole warps and
// elect a lane at each instruction, so that descriptors and coordinates stay in uniform
// registers: issued from a branch that one lane takes, every MMA cost its issuer ~130 cycles.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// D(tmem) (+)= A(smem) * B(smem)^T over the pair, BF16 or FP16 operands, FP32 accumulation;
// issued by one lane of the converged warp.
__device__ __forceinline__ void tc_mma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}

// 32 lanes x 2 consecutive 32-bit columns: thread i of the warp gets lane (base + i).
__device__ __forceinline__ void tmem_ld_32x32b_x2(uint32_t taddr, uint32_t (&r)[2]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr) : "memory");
}

// Shared-memory matrix descriptor of an operand whose rows (the M or N dimension) are
// contiguous: chunks of 64 16-bit values = 128 bytes, one line per reduction step, 128-byte
// swizzle; 8 lines are 1024 bytes, the next 64 values `chunk_bytes` further.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t chunk_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((chunk_bytes >> 4) & 0x3FFFu) << 16;  // leading byte offset
  d |= static_cast<uint64_t>(1024u >> 4) << 32;                    // stride byte offset
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// Two FP32 values to a pair of 16-bit ones.
template <int OUT>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  if constexpr (OUT == kTypeBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Lanes hold feature `lane` of two rows (lo, hi as FP32 bits); each gets two features of one row: an
// even lane its own and the next lane's of the first row, an odd one the lane before's and its
// own of the second.
template <int OUT>
__device__ __forceinline__ uint32_t trade_pair(uint32_t lo, uint32_t hi, float scale, int odd) {
  const uint32_t mine = pack_pair<OUT>(__uint_as_float(lo) * scale, __uint_as_float(hi) * scale);
  const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
  return __byte_perm(mine, other, odd ? 0x3276u : 0x5410u);
}

// Accumulators whose lanes are features and whose columns are rows of the output, stored in rows:
// four warps (one per lane quarter) hold 32 columns of this CTA's 128 features; v: this lane's
// feature in rows row0 .. row0 + 31.  The 32 x 128 values are turned in 8 KB of shared memory and
// leave as whole 256-byte rows (against 64-byte pieces straight from the lanes: 1% less time for the
// grouped products; the 4-bit product is 3 to 9% faster without).  out: 16-byte aligned rows; f0: the
// CTA's first feature, features a multiple of 8; barrier: a named barrier of these four warps.
template <int OUT>
__device__ __forceinline__ void store_turned(const uint32_t (&v)[32], uint8_t* turn, int barrier, int quarter, int lane,
                                             uint16_t* out, int64_t ldo, int row0, int row_end, int f0, int features) {
  asm volatile("bar.sync %0, 128;" ::"r"(barrier) : "memory");  // the stretch before has left
  const int odd = lane & 1;
  uint8_t* to = turn + odd * 256 + ((quarter * 64 + (lane - odd) * 2) ^ (odd << 6));
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    *reinterpret_cast<uint32_t*>(to + j * 256) = trade_pair<OUT>(v[j], v[j + 1], 1.0f, odd);
  }
  asm volatile("bar.sync %0, 128;" ::"r"(barrier) : "memory");
  const int part = lane & 15, f = f0 + part * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = quarter * 8 + i * 2 + (lane >> 4);
    const uint4 q = *reinterpret_cast<const uint4*>(turn + r * 256 + ((part * 16) ^ ((r & 1) << 6)));
    if (row0 + r < row_end && f < features)
      *reinterpret_cast<uint4*>(out + static_cast<int64_t>(row0 + r) * ldo + f) = q;
  }
}

}  // namespace beam
