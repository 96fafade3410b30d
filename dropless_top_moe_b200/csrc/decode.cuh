// Shared pieces of the few-token layer (decode.cu, decode_umma.cu): workspace
// layout, the plan that every block derives from the chosen experts, and the
// ordered work tickets with their bounded waits.
#pragma once

#include "common.cuh"
#include "kernels.cuh"
#include "umma.cuh"

namespace moe {
namespace decode {

constexpr int kMaxTokens = 128;
constexpr int kMaxExperts = 256;
constexpr int kMaskWords = kMaxTokens / 32;
constexpr int kMaxGroups = 32;              // token groups of the router
constexpr uint64_t kTimeoutNs = 2000000000ull;

// Counters, zeroed by the router kernel of every call.
struct Counters {
  int ticket;                  // next unit of work (fp32)
  int abort;                   // a wait gave up: the others stop too
  int done_down;               // finished down-projection work, whole call
  int pad;
  int done_act[kMaxExperts];   // finished pieces of a slot's activations
};

struct Args {
  const void* x;
  const void* W_r;
  const void* W1;
  const void* W3;
  const void* W2;
  int N, H, E, K, F;
  void* y;
  int32_t* top;
  float* weights;
  // workspace
  int* status;
  int* arrive;                 // [kMaxGroups], inside the status region: zero between calls
  int* queue;                  // bf16: next ticket and blocks that have left, zero between calls too
  Counters* cnt;
  int zero_ints;               // the router kernel zeroes this many from cnt on
  float* logit_part;           // [groups][S][TG][E]
  void* act;                   // [N*K][F]
  float* out;                  // [N*K][H]
};

// decode_umma.cu: the expert kernel for bf16
size_t umma_part_bytes(int N);   // partial sums of one phase
moe_status experts_umma(const Args& a, float* part_up, float* part_down, int* tile_cnt, cudaStream_t s);

// ---- plan: which experts are used, by which tokens ---------------------------
// Slots are the used experts in increasing id; a slot's rows are its tokens in
// increasing order.  A token holds an expert at most once, so a bit mask a
// expert says it all, and every block derives the same plan from `top`.
struct Plan {
  uint32_t mask[kMaxExperts][kMaskWords];
  int16_t slot_of[kMaxExperts];
  int16_t expert[kMaxExperts];   // of a slot
  int off[kMaxExperts + 1];      // first row of a slot
  int warp_slots[8], warp_rows[8];
  int slots;
};

// All threads of a block of at least 256.
__device__ __forceinline__ void clear_plan(Plan& p, int threads) {
  for (int i = threadIdx.x; i < kMaxExperts * kMaskWords; i += threads) (&p.mask[0][0])[i] = 0;
  __syncthreads();
}
// After clear_plan, once the router has finished.
__device__ __forceinline__ void build_plan(Plan& p, const int32_t* top, int N, int K, int E, int threads) {
  for (int i = threadIdx.x; i < N * K; i += threads) {
    const int e = __ldcg(top + i), n = i / K;
    if ((unsigned)e < (unsigned)E) atomicOr(&p.mask[e][n >> 5], 1u << (n & 31));
  }
  __syncthreads();
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
  int rows = 0, urows = 0, uslots = 0;
  if (e < kMaxExperts) {
#pragma unroll
    for (int w = 0; w < kMaskWords; ++w) rows += __popc(p.mask[e][w]);
    urows = rows;
    uslots = rows > 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, urows, o), b = __shfl_up_sync(0xffffffffu, uslots, o);
      if (lane >= o) { urows += a; uslots += b; }
    }
    if (lane == 31) { p.warp_rows[warp] = urows; p.warp_slots[warp] = uslots; }
  }
  __syncthreads();
  if (e < kMaxExperts) {
    for (int w = 0; w < warp; ++w) { urows += p.warp_rows[w]; uslots += p.warp_slots[w]; }
    if (rows > 0) {
      p.expert[uslots - 1] = (int16_t)e;
      p.off[uslots - 1] = urows - rows;
    }
    p.slot_of[e] = (int16_t)(uslots - 1);      // of a used expert
    if (e == kMaxExperts - 1) { p.slots = uslots; p.off[uslots] = urows; }
  }
  __syncthreads();
}

// Row of (token n, expert e) among all rows.
__device__ __forceinline__ int plan_row(const Plan& p, int n, int e) {
  int r = p.off[p.slot_of[e]];
#pragma unroll
  for (int w = 0; w < kMaskWords; ++w) {
    const uint32_t m = p.mask[e][w];
    if (w < (n >> 5)) r += __popc(m);
    else if (w == (n >> 5)) r += __popc(m & ((1u << (n & 31)) - 1u));
  }
  return r;
}

// ---- ordered work ----------------------------------------------------------
// Work is handed out in increasing tickets, and a unit only ever waits for
// units with lower tickets.  Those were all taken by blocks that are running,
// and the lowest unfinished one waits for nothing, so the grid makes progress
// whatever number of its blocks is resident: no cooperative launch is needed,
// and two calls on two workspaces may share the GPU.  Every wait is bounded all
// the same.
__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void add_release(int* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// One thread: until *p reaches `want`; false when it gave up.
__device__ __forceinline__ bool wait_count(const int* p, int want, Counters* cnt, int* status) {
  if (ld_acquire(p) >= want) return true;
  const uint64_t t0 = umma::globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (ld_acquire(p) >= want) return true;
    if ((it & 63) == 0) {
      if (*(volatile int*)&cnt->abort) return false;
      if (umma::globaltimer() - t0 > kTimeoutNs) {
        *(volatile int*)&cnt->abort = 1;
        raise_status(status, MOE_DEVERR_TIMEOUT);
        return false;
      }
    }
  }
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace decode
}  // namespace moe
