// The whole MoE layer for a few tokens (a decoding step): router, top-K, the
// selected experts' SwiGLU and the weighted sum, in two launches.
//
//   l = x W_r,  the K largest (ties to the lower id),  w_k = exp(l_k - l_max) / sum_kept,
//   a_{n,k} = silu(x_n W1_e) * (x_n W3_e),  y_n = sum_k w_{n,k} a_{n,k} W2_e.
//
// With one to a few tokens an expert, the time is the reading of the selected
// experts' weights (3 H F elements each), so the weights are read once, with
// no padded copies of tokens and few launches around them.
//
// Router kernel: blocks over slices of H and groups of tokens; each writes its
// slice's partial logits, and the last block of a group to arrive adds the
// slices in order and picks the experts, a warp a token.
//
// Expert kernel (fp32): blocks take tickets in order - gate/up tiles of every
// used expert, then down tiles, then the weighted sums - and wait only for
// lower tickets.  A tile is 16 vectors of columns; 16 groups of threads share the
// rows, 4 tokens at a time, and are added in order, so results have the same
// bits on every run.
#include <math.h>
#include <string.h>

#include "decode.cuh"

namespace moe {
namespace decode {
namespace {

constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteLoads = 16;      // rows of W_r a thread has in flight
constexpr int kRouteRows = kRouteWarps * kRouteLoads;

// V neighbouring elements of a row, as they lie in memory.
template <typename T, int V>
struct Raw {
  static constexpr int B = V * (int)sizeof(T), W = B < 4 ? 1 : B / 4;
  uint32_t w[W];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const T* p) {      // p aligned to B (16 at most)
    if constexpr (B >= 16) {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 v = __ldg((const uint4*)p + i / 4);
        w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
      }
    } else if constexpr (B == 8) {
      const uint2 v = __ldg((const uint2*)p);
      w[0] = v.x; w[1] = v.y;
    } else if constexpr (B == 4) {
      w[0] = __ldg((const uint32_t*)p);
    } else {
      w[0] = __ldg((const uint16_t*)p);
    }
  }
  __device__ __forceinline__ void load_each(const T* p, int n) {   // the first n elements, one by one
    zero();
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) {
        if constexpr (sizeof(T) == 4) w[j] = __ldg((const uint32_t*)p + j);
        else w[j / 2] |= (uint32_t)__ldg((const uint16_t*)p + j) << (16 * (j & 1));
      }
  }
  __device__ __forceinline__ float at(int j) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
    else return j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
  }
};

// A warp takes a row of W_r at a time, V = EP / 32 neighbouring columns a lane, so
// nothing is added across lanes; `wide`: E is a whole number of V columns and a
// lane's are one load.
template <typename T, int TG, int V>
__global__ void __launch_bounds__(kRouteThreads)
decode_route_kernel(const Args a, int S, int wide, int pick) {
  constexpr int EP = 32 * V, cols = TG * EP;
  __shared__ __align__(16) float xs[kRouteRows][TG];
  __shared__ __align__(16) float red[kRouteWarps * cols > 2 * kRouteCols ? kRouteWarps * cols : 2 * kRouteCols];
  __shared__ int last;
  pdl_launch();
  const int tid = threadIdx.x, g = blockIdx.y, s = blockIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const T* x = (const T*)a.x;
  const T* wr = (const T*)a.W_r;
  const int E = a.E, H = a.H;
  const int t0 = g * TG;
  const int nt = a.N - t0 < TG ? a.N - t0 : TG;
  constexpr int XV = Vec<T>::N;                // slices are whole vectors of x
  const int h0 = H / XV * s / S * XV, h1 = H / XV * (s + 1) / S * XV;
  const int c = lane * V;
  float acc[TG][V];
#pragma unroll
  for (int t = 0; t < TG; ++t)
#pragma unroll
    for (int j = 0; j < V; ++j) acc[t][j] = 0.f;
  for (int c0 = h0; c0 < h1; c0 += kRouteRows) {
    const int rows = h1 - c0 < kRouteRows ? h1 - c0 : kRouteRows;
    // the weights' loads go out before x is staged
    Raw<T, V> w[kRouteLoads];
    const T* at = wr + (size_t)(c0 + warp) * E + c;
    if (wide) {
#pragma unroll
      for (int i = 0; i < kRouteLoads; ++i) {
        w[i].zero();
        if (warp + i * kRouteWarps < rows && c < E) w[i].load(at + (size_t)i * kRouteWarps * E);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRouteLoads; ++i)
        w[i].load_each(at + (size_t)i * kRouteWarps * E, warp + i * kRouteWarps < rows ? E - c : 0);
    }
    __syncthreads();
    for (int i = tid; i < rows / XV * TG; i += kRouteThreads) {
      const int t = i % TG, h = i / TG * XV;
      float f[XV];
      Vec<T>::to_float(t < nt ? ld_nc_v4(x + (size_t)(t0 + t) * H + c0 + h) : make_uint4(0, 0, 0, 0), f);
#pragma unroll
      for (int j = 0; j < XV; ++j) xs[h + j][t] = f[j];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRouteLoads; ++i) {
      const int h = warp + i * kRouteWarps;
      if (h < rows) {
#pragma unroll
        for (int t = 0; t < TG; ++t)
#pragma unroll
          for (int j = 0; j < V; ++j) acc[t][j] = fmaf(xs[h][t], w[i].at(j), acc[t][j]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TG; ++t)
#pragma unroll
    for (int j = 0; j < V; ++j) red[warp * cols + t * EP + c + j] = acc[t][j];
  __syncthreads();
  float* part = a.logit_part + (size_t)(g * S + s) * cols;
  for (int i = tid; i < cols; i += kRouteThreads) {
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kRouteWarps; ++q) v += red[q * cols + i];
    part[i] = v;
  }
  if (s == 0 && g == 0)
    for (int i = tid; i < a.zero_ints; i += kRouteThreads) ((int*)a.cnt)[i] = 0;
  for (int64_t i = ((int64_t)g * S + s) * kRouteThreads + tid; i < a.fill_vecs; i += (int64_t)gridDim.y * S * kRouteThreads)
    a.fill[i] = make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);
  if (!pick) return;                  // the expert kernel goes on from here
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    last = atomicAdd(a.arrive + g, 1) == S - 1;
    if (last) a.arrive[g] = 0;        // for the next call
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  pick_experts<V>(a.logit_part + (size_t)g * S * cols, nt, EP, S, cols, E, a.K, red,
                  [&](int t, int k, int e, float w) {
                 const size_t at = (size_t)(t0 + t) * a.K + k;
                 a.top[at] = e;
                 a.weights[at] = w;
               });
}

// ---- experts, one block of 256 threads a tile --------------------------------
constexpr int kThreads = 256;
constexpr int kColThreads = 16, kRowGroups = kThreads / kColThreads;
constexpr int kTM = 4;               // tokens at a time
constexpr int kXRows = 512;          // rows of the tokens' operand staged at a time

// V columns of a weight row from column c on: one 16-byte load, or (rows that
// are not a whole number of vectors long) element by element.
template <typename T, bool WIDE>
__device__ __forceinline__ void load_w(const T* row, int ct, int c0, int cols, float* f) {
  constexpr int V = Vec<T>::N;
  if (WIDE) {
    const int c = c0 + ct * V;
    if (c < cols) {
      Vec<T>::to_float(ld_nc_v4(row + c), f);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = c0 + j * kColThreads + ct;
      f[j] = c < cols ? to_f<T>(row[c]) : 0.f;
    }
  }
}
template <bool WIDE, int V>
__device__ __forceinline__ int tile_col(int ct, int j) {
  return WIDE ? ct * V + j : j * kColThreads + ct;
}

struct Smem {
  Plan plan;
  int tokens[kMaxTokens];
  float xs[kTM][kXRows];
  float red[2][kRowGroups][kColThreads * 8];
  int ticket;
  int ok;
};

// One tile of NM matrices (gate and up, or down) for all tokens of a slot:
// C_m[t][c] = sum_r in[t][r] W_m[r][c]; `in` gives the operand's element, `put`
// takes the NM sums of a (token, column).
template <typename T, bool WIDE, int NM, class In, class Put>
__device__ __forceinline__ void tile(Smem& sm, const T* const (&W)[NM], int depth, int cols, int c0, int cnt, In in,
                                     Put put) {
  constexpr int V = Vec<T>::N, kCols = kColThreads * V;
  const int tid = threadIdx.x, ct = tid % kColThreads, rg = tid / kColThreads;
  for (int t0 = 0; t0 < cnt; t0 += kTM) {
    float acc[kTM][NM][V];
#pragma unroll
    for (int t = 0; t < kTM; ++t)
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[t][m][j] = 0.f;
    for (int r0 = 0; r0 < depth; r0 += kXRows) {
      const int rows = depth - r0 < kXRows ? depth - r0 : kXRows;
      __syncthreads();
      for (int i = tid; i < kTM * kXRows; i += kThreads) {
        const int q = i / kXRows, r = i % kXRows;
        sm.xs[q][r] = t0 + q < cnt && r < rows ? in(t0 + q, r0 + r) : 0.f;
      }
      __syncthreads();
#pragma unroll 4
      for (int r = rg; r < rows; r += kRowGroups) {
        float w[NM][V];
#pragma unroll
        for (int m = 0; m < NM; ++m) load_w<T, WIDE>(W[m] + (size_t)(r0 + r) * cols, ct, c0, cols, w[m]);
#pragma unroll
        for (int t = 0; t < kTM; ++t) {
          const float xv = sm.xs[t][r];
#pragma unroll
          for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int j = 0; j < V; ++j) acc[t][m][j] = fmaf(xv, w[m][j], acc[t][m][j]);
        }
      }
    }
    // the row groups' sums, in order
    for (int t = 0; t < kTM && t0 + t < cnt; ++t) {
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kTM; ++q)
        if (q == t) {
#pragma unroll
          for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int j = 0; j < V; ++j) sm.red[m][rg][tile_col<WIDE, V>(ct, j)] = acc[q][m][j];
        }
      __syncthreads();
      if (tid < kCols && c0 + tid < cols) {
        float v[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          v[m] = 0.f;
#pragma unroll
          for (int q = 0; q < kRowGroups; ++q) v[m] += sm.red[m][q][tid];
        }
        put(t0 + t, c0 + tid, v);
      }
    }
  }
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads)
decode_experts_kernel(const Args a) {
  __shared__ Smem sm;
  constexpr int V = Vec<T>::N, kCols = kColThreads * V;
  const int tid = threadIdx.x;
  const T* x = (const T*)a.x;
  T* act = (T*)a.act;
  clear_plan(sm.plan, kThreads);
  pdl_wait();
  build_plan(sm.plan, a.top, a.N, a.K, a.E, kThreads);
  const int slots = sm.plan.slots;
  const int nft = (int)cdiv(a.F, kCols), nht = (int)cdiv(a.H, kCols);
  const int n_up = slots * nft, n_down = slots * nht;
  const int64_t vecs = (int64_t)a.N * (a.H / V);
  const int n_sum = (int)cdiv(vecs, kThreads);
  for (;;) {
    __syncthreads();
    if (tid == 0) sm.ticket = atomicAdd(&a.cnt->ticket, 1);
    __syncthreads();
    int t = sm.ticket;
    if (t >= n_up + n_down + n_sum) return;
    if (t >= n_up + n_down) {
      // y[n] = sum_k w[n,k] out[row(n,k)], in increasing k
      t -= n_up + n_down;
      if (tid == 0) sm.ok = wait_count(&a.cnt->done_down, n_down, a.cnt, a.status);
      __syncthreads();
      if (!sm.ok) return;
      const int64_t at = (int64_t)t * kThreads + tid;
      if (at < vecs) {
        const int n = (int)(at / (a.H / V)), h = (int)(at % (a.H / V)) * V;
        float s[V];
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = 0.f;
        for (int k = 0; k < a.K; ++k) {
          const int e = __ldcg(a.top + (size_t)n * a.K + k);
          const float w = __ldcg(a.weights + (size_t)n * a.K + k);
          const float* o = a.out + (size_t)plan_row(sm.plan, n, e) * a.H + h;
#pragma unroll
          for (int j = 0; j < V; ++j) s[j] = fmaf(w, __ldcg(o + j), s[j]);
        }
        st_v4((T*)a.y + (size_t)n * a.H + h, Vec<T>::from_float(s));
      }
      continue;
    }
    const bool up = t < n_up;
    if (!up) t -= n_up;
    const int u = up ? t / nft : t / nht;
    const int c0 = (up ? t % nft : t % nht) * kCols;
    const int e = sm.plan.expert[u], base = sm.plan.off[u], cnt = sm.plan.off[u + 1] - base;
    const size_t eo = (size_t)e * a.H * a.F;
    if (up) {
      if (tid < a.N && ((sm.plan.mask[e][tid >> 5] >> (tid & 31)) & 1u))
        sm.tokens[plan_row(sm.plan, tid, e) - base] = tid;
      const T* const W[2] = {(const T*)a.W1 + eo, (const T*)a.W3 + eo};
      tile<T, WIDE, 2>(
          sm, W, a.H, a.F, c0, cnt,
          [&](int r, int h) { return to_f<T>(x[(size_t)sm.tokens[r] * a.H + h]); },
          [&](int r, int c, const float (&v)[2]) { act[(size_t)(base + r) * a.F + c] = from_f<T>(silu_f(v[0]) * v[1]); });
    } else {
      if (tid == 0) sm.ok = wait_count(a.cnt->done_act + u, nft, a.cnt, a.status);
      __syncthreads();
      if (!sm.ok) return;
      const T* const W[1] = {(const T*)a.W2 + eo};
      tile<T, true, 1>(
          sm, W, a.F, a.H, c0, cnt,
          // past L1: another block may have left this sector there half written
          [&](int r, int f) { return to_f<T>(__ldcg(act + (size_t)(base + r) * a.F + f)); },
          [&](int r, int c, const float (&v)[1]) { a.out[(size_t)(base + r) * a.H + c] = v[0]; });
    }
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      add_release(up ? a.cnt->done_act + u : &a.cnt->done_down, 1);
    }
  }
}

// ---- host ------------------------------------------------------------------
inline bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline size_t al256(size_t b) { return (b + 255) & ~(size_t)255; }
inline size_t elem(moe_dtype dt) { return dt == MOE_F32 ? 4 : 2; }

moe_status check(int N, int H, int E, int K, int F, moe_dtype dt) {
  if (dt != MOE_F32 && dt != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (N < 0 || H <= 0 || E <= 0 || K <= 0 || K > E || F <= 0) return MOE_ERR_INVALID_ARG;
  if (N > kMaxTokens || E > kMaxExperts || K > 32) return MOE_ERR_UNSUPPORTED;
  if (dt == MOE_F32 && H % 4 != 0) return MOE_ERR_UNSUPPORTED;
  if (dt == MOE_BF16 && (H % 128 != 0 || F % 128 != 0)) return MOE_ERR_UNSUPPORTED;
  // tile counts, the tensor-core kernel's unit counts and a batch's elements stay within 31 bits
  if (H > (1 << 16) || F > (1 << 16)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The router's cut.  Tokens of a group share the reading of W_r; few tokens
// take a group each, which leaves the last block of a group little to add up.
// Slices of H: enough blocks to fill the GPU twice over, of at least 64 rows.
RouteCut route_cut(int N, int H, int E) {
  RouteCut c;
  c.EP = 32;
  while (c.EP < E) c.EP *= 2;
  c.TG = N <= 8 ? 1 : (N <= 32 ? 2 : 4);
  c.groups = (int)cdiv(N, c.TG);
  const int most = (int)cdiv(H, 64), want = (int)cdiv(296, c.groups);
  c.S = most < want ? most : want;
  return c;
}

size_t part_bytes(int N, int H, int E) {
  // the largest cut of any token count up to N
  size_t most = 0;
  for (int n = 1; n <= N; ++n) {
    const RouteCut c = route_cut(n, H, E);
    const size_t b = (size_t)c.groups * c.S * c.TG * c.EP * sizeof(float);
    if (b > most) most = b;
  }
  return most;
}

// What only the bf16 expert kernel has.
struct UmmaWs {
  int* tile_cnt;
  float* part_up;
  float* part_down;
};

size_t carve(Args* a, UmmaWs* w, char* base, int N, int H, int E, int K, int F, moe_dtype dt) {
  size_t off = kStatusBytes;
  auto take = [&](size_t bytes) {
    char* p = base ? base + off : nullptr;
    off += al256(bytes);
    return (void*)p;
  };
  const int64_t used = (int64_t)N * K < E ? (int64_t)N * K : E;
  const size_t tiles = dt == MOE_BF16 ? (size_t)used * (F / 128) : 0;
  const size_t zero = sizeof(Counters) + tiles * sizeof(int);
  void* cnt = take(zero);
  void* part = take(part_bytes(N, H, E));
  // the direct variant's activations are fp32
  const size_t act_row = (size_t)K * F * elem(dt);
  const size_t direct_rows = (size_t)(N < kDirectTokens ? N : kDirectTokens) * K * F * sizeof(float);
  const size_t fill0 = off;
  void* act = take(dt == MOE_BF16 && direct_rows > N * act_row ? direct_rows : N * act_row);
  void* out = take((size_t)N * K * H * sizeof(float));
  void* pu = dt == MOE_BF16 ? take(umma_up_bytes(N, H, E, K, F)) : nullptr;
  void* pd = dt == MOE_BF16 ? take(umma_down_bytes(N, H, E, K, F)) : nullptr;
  if (a) {
    a->status = (int*)base;
    a->arrive = (int*)(base + 64);
    a->queue = (int*)(base + 192);
    a->cnt = (Counters*)cnt;
    a->zero_ints = (int)(zero / sizeof(int));
    if (dt == MOE_BF16 && N <= kDirectTokens) {
      a->fill = (uint4*)act;
      a->fill_vecs = (int64_t)((off - fill0) / sizeof(uint4));
    }
    w->tile_cnt = (int*)((char*)cnt + sizeof(Counters));
    w->part_up = (float*)pu;
    w->part_down = (float*)pd;
    a->logit_part = (float*)part;
    a->act = act;
    a->out = (float*)out;
  }
  return off;
}

template <typename T, int TG>
void route(const Args& a, const RouteCut& c, int pick, cudaStream_t s) {
  const dim3 grid(c.S, c.groups);
  const int wide = a.E % (c.EP / 32) == 0;
#define MOE_DECODE_ROUTE(V)                                                                                    \
  case 32 * V:                                                                                                 \
    MOE_TRACED("decode_route", s,                                                                              \
               (decode_route_kernel<T, TG, V><<<grid, kRouteThreads, 0, s>>>(a, c.S, wide, pick)));            \
    break;
  switch (c.EP) {
    MOE_DECODE_ROUTE(1)
    MOE_DECODE_ROUTE(2)
    MOE_DECODE_ROUTE(4)
    MOE_DECODE_ROUTE(8)
  }
#undef MOE_DECODE_ROUTE
}

template <typename T>
moe_status route_any(const Args& a, const RouteCut& c, int pick, cudaStream_t s) {
  if (c.TG == 1) route<T, 1>(a, c, pick, s);
  else if (c.TG == 2) route<T, 2>(a, c, pick, s);
  else route<T, 4>(a, c, pick, s);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

// Launched while the router still runs: it waits there for the router's end.
template <class Kernel>
moe_status launch_after(Kernel k, int blocks, int threads, const Args& a, cudaStream_t s, const char* name) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t err = cudaSuccess;
  MOE_TRACED(name, s, (err = cudaLaunchKernelEx(&cfg, k, a)));
  if (err != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

template <typename T>
moe_status experts(const Args& a, cudaStream_t s) {
  const int blocks = 148 * 4;
  return a.F % Vec<T>::N == 0 ? launch_after(decode_experts_kernel<T, true>, blocks, kThreads, a, s, "decode_experts")
                              : launch_after(decode_experts_kernel<T, false>, blocks, kThreads, a, s, "decode_experts");
}

}  // namespace
}  // namespace decode
}  // namespace moe

using namespace moe;

extern "C" {

int32_t moe_decode_max_tokens(void) { return decode::kMaxTokens; }

size_t moe_layer_decode_workspace_size(int32_t N, int32_t H, int32_t E, int32_t K, int32_t F, moe_dtype dt) {
  if (decode::check(N, H, E, K, F, dt) != MOE_OK) return 0;
  return decode::carve(nullptr, nullptr, nullptr, N, H, E, K, F, dt);
}

moe_status moe_layer_decode(const void* x, const void* W_r, const void* W1, const void* W3, const void* W2,
                            int32_t N, int32_t H, int32_t E, int32_t K, int32_t F, moe_dtype dt, void* y,
                            int32_t* top_experts, float* weights, void* ws, size_t ws_bytes, moe_stream_t stream) {
  using namespace decode;
  const moe_status st = check(N, H, E, K, F, dt);
  if (st != MOE_OK) return st;
  if (!W_r || !W1 || !W3 || !W2 || (N > 0 && (!x || !y || !top_experts || !weights))) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {x, W_r, W1, W3, W2, y, top_experts, weights, ws};
  for (const void* p : ptrs)
    if (!al16(p)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < moe_layer_decode_workspace_size(N, H, E, K, F, dt)) return MOE_ERR_WORKSPACE;
  if (N == 0) return MOE_OK;
  Args a;
  memset(&a, 0, sizeof(a));
  a.x = x; a.W_r = W_r; a.W1 = W1; a.W3 = W3; a.W2 = W2;
  a.N = N; a.H = H; a.E = E; a.K = K; a.F = F;
  a.y = y; a.top = top_experts; a.weights = weights;
  UmmaWs w;
  carve(&a, &w, (char*)ws, N, H, E, K, F, dt);
  cudaStream_t s = (cudaStream_t)stream;
  const RouteCut c = route_cut(N, H, E);
  if (dt == MOE_F32) {
    const moe_status rs = route_any<float>(a, c, 1, s);
    return rs != MOE_OK ? rs : experts<float>(a, s);
  }
  const moe_status rs = route_any<__nv_bfloat16>(a, c, N > kPickTokens, s);
  return rs != MOE_OK ? rs : experts_umma(a, c, w.part_up, w.part_down, w.tile_cnt, s);
}

}  // extern "C"
