// Diagnostics: the bounded pipeline wait on a barrier that never completes.
//
// Every mbarrier wait of the tcgen05 GEMM pipelines is bounded: after a time
// limit the waiting thread raises the kernel's abort flag, sets
// MOE_DEVERR_TIMEOUT in the caller's status word and returns, so a stalled
// pipeline ends the kernel with an error the host can read instead of hanging
// the GPU.  moe_selftest_wait_timeout runs that same wait (mbar_wait_bounded)
// in one block on a barrier nothing ever arrives at, with a caller-chosen
// limit, so the failure path can be exercised without a fault.
// moe_selftest_handover_timeout does the same for the few-token layer's waits on
// values that other blocks hand over.
#include "common.cuh"
#include "decode.cuh"
#include "kernels.cuh"
#include "umma.cuh"

namespace {

using namespace moe::umma;

__global__ void wait_timeout_kernel(int* status, uint64_t timeout_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    fence_barrier_init();
    abort_flag = 0;
  }
  __syncthreads();
  // one arrival expected, none made: only the time limit ends this wait
  if (threadIdx.x == 0) (void)mbar_wait_bounded(smem_u32(&bar), 0, &abort_flag, status, timeout_ns);
}

// One thread: a counter that stays below what is waited for, the same wait once another has given up, and a
// word that stays empty.
__global__ void handover_timeout_kernel(moe::decode::Counters* cnt, float* word, int* status, uint64_t limit,
                                        int32_t* seen) {
  using namespace moe::decode;
  volatile int* abort = &cnt->abort;
  int bits = 0;
  *abort = 0;
  *(volatile int*)&cnt->done_act[0] = 0;
  *(volatile uint32_t*)word = kEmpty;
  if (!wait_count(&cnt->done_act[0], 1, cnt, status, limit) && *abort) bits |= 1;
  if (!wait_count(&cnt->done_act[0], 1, cnt, nullptr, 1000 * limit)) bits |= 2;     // ended by abort, long before
  *abort = 0;
  Patience patience;
  patience.limit = limit;
  float v = ld_word(word);
  while (__float_as_uint(v) == kEmpty && patience.again(cnt, status)) v = ld_word(word);
  if (__float_as_uint(v) == kEmpty && *abort) bits |= 4;
  *seen = bits;
}

}  // namespace

extern "C" moe_status moe_selftest_handover_timeout(void* ws, size_t ws_bytes, int64_t timeout_ns, int32_t* seen,
                                                    moe_stream_t stream) {
  using namespace moe;
  if (!ws || ((uintptr_t)ws & 15u) || !seen || timeout_ns < 1000 || timeout_ns > 1000000000) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < kStatusBytes + sizeof(decode::Counters) + sizeof(float)) return MOE_ERR_WORKSPACE;
  decode::Counters* cnt = (decode::Counters*)((char*)ws + kStatusBytes);
  cudaStream_t s = (cudaStream_t)stream;
  MOE_TRACED("selftest_handover_timeout", s,
             (handover_timeout_kernel<<<1, 1, 0, s>>>(cnt, (float*)(cnt + 1), (int*)ws, (uint64_t)timeout_ns, seen)));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

extern "C" moe_status moe_selftest_wait_timeout(int32_t* status, int64_t timeout_ns, moe_stream_t stream) {
  if (!status || timeout_ns < 1000 || timeout_ns > 1000000000) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  MOE_TRACED("selftest_wait_timeout", s, (wait_timeout_kernel<<<1, 32, 0, s>>>((int*)status, (uint64_t)timeout_ns)));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}
