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

// One CTA waits, with the operators' bounded wait, at a barrier that nothing completes.
__global__ void operators_timeout_probe_kernel(uint64_t limit_ns, uint32_t* grouped, uint32_t* fp4, int32_t* result) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
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
  }
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
  if (limit_ns <= 0 || limit_ns > static_cast<int64_t>(kWaitLimitNs) || !result ||
      (reinterpret_cast<uintptr_t>(result) & 3))
    return BEAM_MOE_ERR_INVALID_ARG;
  uint32_t *grouped = nullptr, *fp4 = nullptr;
  cudaError_t e = grouped_gemm_error_word(&grouped);
  if (e == cudaSuccess) e = gemm_fp4_error_word(&fp4);
  if (e != cudaSuccess) return BEAM_MOE_ERR_CUDA;
  operators_timeout_probe_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<uint64_t>(limit_ns),
                                                                                  grouped, fp4, result);
  return cudaGetLastError() == cudaSuccess ? BEAM_MOE_OK : BEAM_MOE_ERR_CUDA;
}

}  // extern "C"
