// What the operators on caller buffers share on the host: their error words (they have no
// handle), and a probe that makes their waits run out.
#include <mutex>

#include "../../include/beam_moe.h"
#include "cta_pair.cuh"
#include "internal.h"

namespace beam {

namespace {

__device__ uint32_t g_taken;  // what the last check found, under g_check_mutex
std::mutex g_check_mutex;

// Reads and clears in one step, so that a bit set meanwhile by a kernel of another stream is either
// in this check's answer or in the next one's.
__global__ void take_errors_kernel(uint32_t* grouped, uint32_t* fp4) {
  g_taken = atomicExch(grouped, 0u) | atomicExch(fp4, 0u);
}

// One CTA waits, with the operators' bounded wait, at a barrier that nothing completes (result[0]).
// Then its second warp waits at a barrier that the first completes after three limits, making
// progress in between, and once more, without progress, at the other one (result[3]: met, not met).
__global__ void operators_timeout_probe_kernel(uint64_t limit_ns, uint32_t* grouped, uint32_t* fp4, int32_t* result) {
  __shared__ uint64_t bar, later;
  __shared__ int abort_flag;
  __shared__ uint32_t progress;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    mbar_init(&later, 1);
    abort_flag = 0;
    progress = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const bool gave_up = !pair_wait(&bar, 0, &abort_flag, limit_ns);
  __syncthreads();
  if (threadIdx.x == 0) {
    result[0] = gave_up && abort_flag;
    if (abort_flag) {
      atomicOr(grouped, kErrTimeoutMma);
      atomicOr(fp4, kErrTimeoutMma);
    }
    abort_flag = 0;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (uint32_t i = 1; i <= 12; ++i) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < limit_ns / 4) __nanosleep(1000);
      *static_cast<volatile uint32_t*>(&progress) = i;
    }
    mbar_arrive_at(map_to_cta(&later, 0));
  } else if (threadIdx.x == 32) {
    const bool met = pair_wait(&later, 0, &abort_flag, limit_ns, &progress);
    result[3] = met && !pair_wait(&bar, 0, &abort_flag, limit_ns, &progress) && abort_flag;
  }
}

// A cluster of two CTAs hands sums over as the pairs of a shared tile do.
//   late: the receiver has given up, the sender sends two limits later: the receiver must still be
//         there when the sums land (result: they had, and it reports that it gave up);
//   else: the sender's own wait gives up: the receiver is released by it, well before its own limit.
constexpr uint32_t kProbeWords = 512;
__global__ void sums_probe_kernel(uint64_t limit_ns, int late, int32_t* result) {
  __shared__ alignas(16) uint32_t sums[kProbeWords];
  __shared__ uint64_t bar, never;
  __shared__ int abort_flag;
  const uint32_t rank = cluster_cta_rank();
  pdl_wait();
  for (uint32_t i = threadIdx.x; i < kProbeWords; i += blockDim.x) sums[i] = rank == 0 ? 0u : i + 1;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    mbar_init(&never, 1);
    abort_flag = rank == 0 && late;
    if (rank == 0) mbar_arrive_expect_tx(&bar, kProbeWords * 4);
    fence_mbar_init();
  }
  fence_proxy_async_smem();
  __syncthreads();
  cluster_sync();
  if (rank == 1) {
    bool ok = late != 0;
    if (late) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2 * limit_ns) __nanosleep(1000);
    } else {
      ok = __all_sync(0xffffffffu, pair_wait(&never, 0, &abort_flag, limit_ns));
    }
    __syncwarp();
    if (threadIdx.x == 0) send_sums(ok, map_to_cta(sums, 0), sums, kProbeWords * 4, map_to_cta(&bar, 0));
  } else {
    const bool got = receive_sums(!late, &bar, &abort_flag, kWaitLimitNs);
    bool right = got != (late != 0);
    if (late)
      for (uint32_t i = threadIdx.x; i < kProbeWords; i += blockDim.x) right = right && sums[i] == i + 1;
    right = __all_sync(0xffffffffu, right);
    if (threadIdx.x == 0) *result = right;
  }
  __syncwarp();
  cluster_sync();
}

}  // namespace

}  // namespace beam

using namespace beam;

extern "C" {

beam_moe_status beam_moe_check_operators(void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const std::lock_guard<std::mutex> lock(g_check_mutex);
  uint32_t *grouped = nullptr, *fp4 = nullptr, bits = 0;
  cudaError_t e = grouped_gemm_error_word(&grouped);
  if (e == cudaSuccess) e = gemm_fp4_error_word(&fp4);
  if (e != cudaSuccess) return BEAM_MOE_ERR_CUDA;
  take_errors_kernel<<<1, 1, 0, s>>>(grouped, fp4);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(&bits, g_taken, sizeof(bits), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return BEAM_MOE_ERR_CUDA;
  return bits ? BEAM_MOE_ERR_TIMEOUT : BEAM_MOE_OK;
}

beam_moe_status beam_moe_debug_operators_timeout(int64_t limit_ns, int32_t* result, void* stream) {
  if (limit_ns <= 0 || limit_ns > static_cast<int64_t>(kWaitLimitNs / 4) || !result ||
      !aligned_to(result, 4))
    return BEAM_MOE_ERR_INVALID_ARG;
  uint32_t *grouped = nullptr, *fp4 = nullptr;
  cudaError_t e = grouped_gemm_error_word(&grouped);
  if (e == cudaSuccess) e = gemm_fp4_error_word(&fp4);
  if (e != cudaSuccess) return BEAM_MOE_ERR_CUDA;
  operators_timeout_probe_kernel<<<1, 64, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<uint64_t>(limit_ns),
                                                                                  grouped, fp4, result);
  e = cudaGetLastError();
  for (int late = 0; late < 2 && e == cudaSuccess; ++late)
    e = launch_pdl_clusters(sums_probe_kernel, 2, 2, 32, 0, static_cast<cudaStream_t>(stream),
                            static_cast<uint64_t>(limit_ns), late, result + 1 + late);
  return launch_status(e);
}

}  // extern "C"
