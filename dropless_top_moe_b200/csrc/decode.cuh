// Shared pieces of the few-token layer (decode.cu, decode_umma.cu): workspace
// layout, the plan that every block derives from the chosen experts, and the
// ordered work tickets with their bounded waits.
#pragma once

#include "common.cuh"
#include "decode_line.cuh"
#include "kernels.cuh"
#include "pdl.cuh"
#include "umma.cuh"

#include <math.h>

namespace moe {
namespace decode {

constexpr int kMaxTokens = 128;
static_assert(kMaxTokens <= kBlocks, "a block's share of y lies in two rows");
constexpr int kMaxExperts = 256;
constexpr int kMaskWords = kMaxTokens / 32;
constexpr int kMaxGroups = 32;              // token groups of the router
constexpr uint64_t kTimeoutNs = 2000000000ull;

// Counters, zeroed by the router kernel of every call.
struct Counters {
  int abort;                   // a wait gave up: the others stop too
  int done_down;               // finished down-projection work, whole call
  int pad[2];
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
  int* queue;                  // next ticket and blocks that have left, zero between calls too
  Counters* cnt;
  uint4* fill;                 // words that the router kernel sets to all ones
  int64_t fill_vecs;
  int zero_ints;               // the router kernel zeroes this many from cnt on
  float* logit_part;           // [groups][S][TG][E]
  void* act;                   // fp32 [N*K][F], or bf16 [2][N*K][F] (decode_umma.cu)
  float* out;                  // [N*K][H]
};

// ---- router ------------------------------------------------------------------
// The router kernel leaves partial logits of slices of H, in groups of TG tokens:
// logit_part[group][slice][token of the group][EP columns].
constexpr int kRouteThreads = 256;
constexpr int kRouteCols = 1024;     // most (token, expert) sums of a group
// With few partial logits (kPickTokens tokens, kPickFloats values) every block of the
// expert kernel picks the experts itself, rather than wait for the router's last block to do
// it and read the result; with more they would read more than they save.
constexpr int kPickTokens = 8;       // the router's groups are of one token up to here (route_cut)
constexpr int kPickFloats = 8192;
struct RouteCut {
  int TG, groups, S, EP;
  bool here;           // the expert kernel picks
};

// Order of floats as unsigned numbers; NaN ranks like -infinity.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(isnan(v) ? -INFINITY : v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A block of kRouteThreads threads or more: the experts and weights of `rows` tokens, at most 8 and
// at most kRouteCols / EP, EP = 32 V.  Slice q's partial logits of row r start at
// all + r * row_stride + q * slice_stride; they are added in order.
// put(row, k, id, weight).  red: 2 * kRouteCols floats.
template <int V, class Put>
__device__ __forceinline__ void pick_experts(const float* all, int rows, size_t row_stride, int S,
                                             size_t slice_stride, int E, int K, float* red, Put put) {
  constexpr int EP = 32 * V, QV = EP / 4;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int lc = __ffs(QV) - 1;                     // log2 of the vectors of all rows
  while ((1 << lc) < rows * QV) ++lc;
  const int CV = 1 << lc, SL = kRouteThreads >> lc, cols = CV * 4;   // SL threads add up four columns
  {
    const int cv = tid & (CV - 1), sl = tid >> lc, r = cv / QV;
    const float* at = all + r * row_stride + (cv % QV) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows && tid < kRouteThreads) {
      for (int q = sl; q < S; q += 8 * SL) {        // eight slices in flight
        float4 o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = q + i * SL < S ? __ldcg((const float4*)(at + (q + i * SL) * slice_stride))
                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) { v.x += o[i].x; v.y += o[i].y; v.z += o[i].z; v.w += o[i].w; }
      }
    }
    for (int o = CV; o < 32; o <<= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
      v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
    }
    const int lines = CV < 32 ? kRouteThreads / 32 : SL;
    if (tid < kRouteThreads && (CV >= 32 || lane < CV)) ((float4*)red)[(CV < 32 ? warp : sl) * CV + cv] = v;
    __syncthreads();
    for (int i = tid; i < cols; i += kRouteThreads) {
      float t = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) t += q < lines ? red[q * cols + i] : 0.f;
      red[kRouteCols + i] = t;
    }
    __syncthreads();
  }
  if (warp >= rows) return;
  const float* lg = red + kRouteCols + warp * EP;
  // K rounds of arg-max over (value, id): the keys order totally and 0 marks
  // one already taken, so the ids stay distinct
  uint32_t key[V];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 32 + lane;
    key[i] = e < E ? order_key(lg[e]) : 0u;
    if (e < E) m = fmaxf(m, lg[e]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  int my_id = 0;
  for (int k = 0; k < K; ++k) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = key[i] > best ? key[i] : best;
    best = __reduce_max_sync(0xffffffffu, best);
    uint32_t id = 0xffffffffu;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (key[i] == best) id = (uint32_t)(i * 32 + lane);
    id = __reduce_min_sync(0xffffffffu, id);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (id == (uint32_t)(i * 32 + lane)) key[i] = 0u;
    if (lane == k) my_id = (int)id;
  }
  const float ek = lane < K ? expf(lg[my_id] - m) : 0.f;
  const float Z = warp_sum(ek);
  if (lane < K) put(warp, lane, my_id, ek / Z);
}

// ---- decode_umma.cu: the expert kernel for bf16 --------------------------------
// Up to this many tokens its blocks hand partial sums and fp32 activations over
// without flags (1 token 2048/64/6/1408: 36 us with flags, 30 without; 4 tokens: 84, 74;
// 7 tokens: 100, 105).
constexpr int kDirectTokens = 4;
size_t umma_up_bytes(int N, int H, int E, int K, int F);     // partial sums of gate and up
size_t umma_down_bytes(int N, int H, int E, int K, int F);   // of the down product
moe_status experts_umma(const Args& a, const RouteCut& cut, float* part_up, float* part_down, int* tile_cnt,
                        cudaStream_t s);

// ---- values that are their own flags --------------------------------------------
// The router kernel fills a buffer with a NaN that no sum has; readers poll the
// words that they need.  A word holds all that a reader asks of it, so nothing
// else has to be ordered.
constexpr uint32_t kEmpty = 0xffffffffu;
__device__ __forceinline__ float not_empty(float v) {
  return __float_as_uint(v) == kEmpty ? __uint_as_float(0x7fffffffu) : v;
}
__device__ __forceinline__ void st_word(float* p, float v) {
  asm volatile("st.relaxed.gpu.global.f32 [%0], %1;" ::"l"(p), "f"(not_empty(v)) : "memory");
}
__device__ __forceinline__ float ld_word(const float* p) {
  float v;
  asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_words2(const float* p) {
  float2 v;
  asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_words4(const float* p) {
  float4 v;
  asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ bool empty(float2 v) {
  return __float_as_uint(v.x) == kEmpty || __float_as_uint(v.y) == kEmpty;
}
__device__ __forceinline__ bool empty(float4 v) {
  return __float_as_uint(v.x) == kEmpty || __float_as_uint(v.y) == kEmpty || __float_as_uint(v.z) == kEmpty ||
         __float_as_uint(v.w) == kEmpty;
}
// The limit of a thread that polls words.
struct Patience {
  uint64_t t0 = 0, limit = kTimeoutNs;
  uint32_t it = 0;
  // another look: false when this thread, or another, gave up
  __device__ __forceinline__ bool again(Counters* cnt, int* status) {
    if ((++it & 63) != 0) return true;
    if (*(volatile int*)&cnt->abort) return false;
    const uint64_t now = umma::globaltimer();
    if (t0 == 0) t0 = now;
    if (now - t0 <= limit) return true;
    *(volatile int*)&cnt->abort = 1;
    raise_status(status, MOE_DEVERR_TIMEOUT);
    return false;
  }
};

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
__device__ __forceinline__ void plan_add(Plan& p, int n, int e) { atomicOr(&p.mask[e][n >> 5], 1u << (n & 31)); }
// After clear_plan, once the ids are there: from the router's output, or (top
// NULL) added with plan_add.
__device__ __forceinline__ void build_plan(Plan& p, const int32_t* top, int N, int K, int E, int threads) {
  if (top)
    for (int i = threadIdx.x; i < N * K; i += threads) {
      const int e = __ldcg(top + i);
      if ((unsigned)e < (unsigned)E) plan_add(p, i / K, e);
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

// What a block of the expert kernel picked, for cut.here.
struct Picked {
  int id[kPickTokens][32];
  float w[kPickTokens][32];
};
template <int V>
__device__ __forceinline__ void pick_all_v(const Args& a, const RouteCut& cut, Plan& plan, Picked& pick, float* red) {
  constexpr int EP = 32 * V;
  const int pass = kRouteCols / EP < kPickTokens ? kRouteCols / EP : kPickTokens;
  for (int n0 = 0; n0 < a.N; n0 += pass) {
    if (n0) __syncthreads();
    pick_experts<V>(a.logit_part + (size_t)n0 * cut.S * EP, a.N - n0 < pass ? a.N - n0 : pass, (size_t)cut.S * EP,
                    cut.S, EP, a.E, a.K, red, [&](int r, int k, int e, float w) {
                      const int n = n0 + r;
                      plan_add(plan, n, e);
                      pick.id[n][k] = e;
                      pick.w[n][k] = w;
                      if (blockIdx.x == 0) {
                        a.top[n * a.K + k] = e;
                        a.weights[n * a.K + k] = w;
                      }
                    });
  }
}
// After clear_plan; the router's groups are of one token.
__device__ __forceinline__ void pick_all(const Args& a, const RouteCut& cut, Plan& plan, Picked& pick, float* red) {
  switch (cut.EP) {
    case 32: pick_all_v<1>(a, cut, plan, pick, red); break;
    case 64: pick_all_v<2>(a, cut, plan, pick, red); break;
    case 128: pick_all_v<4>(a, cut, plan, pick, red); break;
    default: pick_all_v<8>(a, cut, plan, pick, red); break;
  }
}

// A block's share of y: vectors [v0, v1) of four columns.  At most a row, so it lies in one
// or two tokens (kMaxTokens <= kBlocks).
struct Share {
  int per_row, v0, v1, first;
};
__device__ __forceinline__ Share share_of(const Args& a, int blocks) {
  Share h;
  h.per_row = a.H / 4;
  const int vecs = a.N * h.per_row, share = (vecs + blocks - 1) / blocks;
  h.v0 = (int)blockIdx.x * share;
  h.v1 = h.v0 + share < vecs ? h.v0 + share : vecs;
  h.first = h.v0 / h.per_row;
  return h;
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
__device__ __forceinline__ bool wait_count(const int* p, int want, Counters* cnt, int* status,
                                           uint64_t limit = kTimeoutNs) {
  if (ld_acquire(p) >= want) return true;
  const uint64_t t0 = umma::globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (ld_acquire(p) >= want) return true;
    if ((it & 63) == 0) {
      if (*(volatile int*)&cnt->abort) return false;
      if (umma::globaltimer() - t0 > limit) {
        *(volatile int*)&cnt->abort = 1;
        raise_status(status, MOE_DEVERR_TIMEOUT);
        return false;
      }
    }
  }
}

}  // namespace decode
}  // namespace moe
