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
// slices in order and picks the experts, a warp a token; with few logits the expert
// kernel's blocks each do that themselves.  It also clears what the expert kernel
// hands values over in.  5 us for 33 tokens (2048 x 64), most of it latency: the loads of
// W_r and x, a counter's round trip, the slices' sums, K rounds of arg-max.
//
// Expert kernels: below for fp32, decode_umma.cu for bf16.
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
  auto fill = [&]() {
    const int64_t all = (int64_t)gridDim.y * gridDim.x * kRouteThreads;
    for (int64_t i = ((int64_t)g * gridDim.x + s) * kRouteThreads + tid; i < a.fill_vecs; i += all)
      a.fill[i] = make_uint4(kEmpty, kEmpty, kEmpty, kEmpty);
  };
  if (s >= S) {                 // a block past the slices: there to fill
    fill();
    return;
  }
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
  fill();
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

// ---- fp32 experts ------------------------------------------------------------
// fp32 layers keep full single precision, so their products are FMAs.  A block
// takes a tile of 4 CT columns (gate and up of the same ones; down has a CT of its own), its 256 / CT
// row groups take the rows in turn, TM tokens share each weight, and the groups'
// sums are added in a fixed order.  Every thread copies its own weights to shared
// memory kAhead rows ahead (cp.async): they keep coming across the barriers around the
// tokens' staging, and need no barrier themselves.  Activations and expert outputs are
// handed over as words that are their own flags, tiles as tickets in order, so
// the phases run into each other.  HBM bounds it with few tokens an expert; beyond, every
// chunk of kTokens tokens passes over its expert's weights again, from L2, and nothing is full:
// 50 tokens 824/33/7/918 (142 us, floor 46) keep 15 warps an SM that issue in 52 % of the
// cycles, the FMA pipe 34 % busy, DRAM 28 %.
constexpr int kThreads = 256;
constexpr int kXRows = 512;          // rows of the tokens' operand staged at a time
constexpr int kTokens = 8;           // most tokens at a time
constexpr int kAhead = 8;            // rows of a thread under way or in hand

constexpr int kRingVec = 320;        // 16-byte vectors of one row of every row group, one matrix

template <int CT, bool WIDE>
__device__ __forceinline__ int tile_col(int ct, int j) {
  return WIDE ? ct * 4 + j : j * CT + ct;
}
// 16 bytes to shared memory, of which the first `bytes` are read and the rest are zero.
__device__ __forceinline__ void copy_async(void* dst, const void* src, int bytes = 16) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}

// two sums in one instruction: c = a * b + c, each rounded as fmaf's (1 to 4 % of a layer's time,
// most with many tokens an expert)
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ void fma2(uint64_t& c, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}

struct Smem {
  Plan plan;
  Picked pick;
  int chunk0[kMaxExperts + 1];       // token chunks of kTokens before a slot's
  int tokens[kMaxTokens];
  int ticket;
  alignas(16) float xs[kXRows * kTokens];        // [row][token]
  // the weights under way, [row][matrix][...]; then a tile's sums, [warp][token][matrix][column]
  alignas(16) float4 ring[kAhead * 2 * kRingVec];
};
static_assert(sizeof(((Smem*)0)->ring) >= 2 * kRouteCols * sizeof(float), "pick_experts' scratch");
static_assert(sizeof(((Smem*)0)->ring) >= 8 * kTokens * 2 * 64 * sizeof(float), "a tile's sums");

// A tile of NM matrices for TM tokens from row t0 of a slot on:
// C_m[t][c] = sum_r in(t)[r] W_m[r][c]; put(t, c, sums) takes them.  POLL: the words that
// `in` points to may still be empty.  Those of x are not read through the read-only path: y may be written
// over x, by blocks that are done with a token, while others still read.
template <int CT, bool WIDE, bool POLL, int NM, int TM, class In, class Put>
__device__ __forceinline__ void tile_tokens(const Args& a, Patience& patience, Smem& sm, const float* const (&W)[NM],
                                            int depth, int cols, int c0, int t0, int cnt, In in, Put put) {
  constexpr int RG = kThreads / CT, C = 4 * CT;
  const int tid = threadIdx.x, ct = tid % CT, rg = tid / CT, warp = tid >> 5, lane = tid & 31;
  // WIDE: every thread copies, and reads, its own vector.  Else a row starts anywhere
  // in a vector: a row group's CT lanes copy the CT + 1 aligned vectors that cover its
  // columns (what lies past the matrix's end is not read) and read each other's, PITCH
  // floats a row group so that a warp's reads meet no bank twice.
  constexpr int PITCH = WIDE ? C : (CT == 4 ? 20 : C + (CT == 8 ? 8 : 16));
  static_assert(RG * PITCH <= kRingVec * 4, "a row of the ring");
  const int warp_rg = warp * 32 / CT;                    // the warp's first row group
  // A thread's rows are RG apart, and RG is a multiple of 4: where its columns start in
  // an aligned vector, and so what each of its copies takes, is the same in every row.
  constexpr int SLOT = NM * kRingVec * 16;               // bytes of a row of every row group
  static_assert(RG % 4 == 0, "a thread's rows start alike");
  const float* src[NM];                                  // the thread's vector of the next row to ask for
  int own[NM], tail[NM];                                 // bytes of it, and of the vector past the CT-th
  int at[NM];                                            // where in a slot the thread reads
#pragma unroll
  for (int m = 0; m < NM; ++m) {
    const float* p = W[m] + (size_t)rg * cols + c0;
    const int lead = WIDE ? 0 : (int)(((uintptr_t)p >> 2) & 3u);        // elements before the first column
    const int need = lead + (cols - c0 < C ? cols - c0 : C);            // from the aligned start on
    const int mine = need - ct * 4, past = need - C;
    src[m] = p - lead + ct * 4;
    own[m] = mine < 0 ? 0 : (mine < 4 ? mine * 4 : 16);
    tail[m] = ct == 0 && past > 0 ? past * 4 : 0;
    at[m] = (m * kRingVec * 4 + rg * PITCH + (WIDE ? ct * 4 : lead + ct)) * (int)sizeof(float);
  }
  char* const mine = (char*)sm.ring + (rg * PITCH + ct * 4) * sizeof(float);     // where in a slot it copies to
  const size_t step = (size_t)RG * cols;
  auto ask = [&](int i) {
    if (rg + i * RG < depth) {
      char* dst = mine + (i % kAhead) * SLOT;
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        if (WIDE) {
          if (own[m] > 0) copy_async(dst + m * kRingVec * 16, src[m]);
        } else {
          if (own[m] > 0) copy_async(dst + m * kRingVec * 16, src[m], own[m]);
          if (tail[m] > 0) copy_async(dst + m * kRingVec * 16 + CT * 16, src[m] + C, tail[m]);
        }
        src[m] += step;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i) ask(i);
  uint64_t acc[TM][NM][2];               // columns 0 and 1, 2 and 3 of the thread's
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[t][m][j] = 0;
  int i = 0;
  for (int r0 = 0; r0 < depth; r0 += kXRows) {
    const int rows = depth - r0 < kXRows ? depth - r0 : kXRows;
    __syncthreads();
    // a warp reads eight rows (32 bytes) of four tokens, whose words meet few banks twice;
    // eight loads of a thread in flight
    constexpr int XT = TM < 4 ? TM : 4, STEP = kThreads / TM;
    const int t = lane % XT + XT * (warp % (TM / XT)), first = lane / XT + 32 / XT * (warp / (TM / XT));
    if (t0 + t < cnt) {
      const float* row = in(t0 + t) + r0;
      for (int e0 = first; e0 < rows; e0 += 8 * STEP) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = 0.f;
          if (e0 + j * STEP < rows) v[j] = POLL ? ld_word(row + e0 + j * STEP) : row[e0 + j * STEP];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (e0 + j * STEP >= rows) break;
          if (POLL)
            while (__float_as_uint(v[j]) == kEmpty && patience.again(a.cnt, a.status)) v[j] = ld_word(row + e0 + j * STEP);
          sm.xs[(e0 + j * STEP) * TM + t] = v[j];
        }
      }
    }
    __syncthreads();
    for (; warp_rg + i * RG < r0 + rows; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
      if (!WIDE) __syncwarp();          // the other lanes' copies are here, and their reads of the last turn done
      const int r = rg + i * RG;
      const char* slot = (const char*)sm.ring + (i % kAhead) * SLOT;
      float4 w[NM];
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const float* in_slot = (const float*)(slot + at[m]);
        if (WIDE)
          w[m] = *(const float4*)in_slot;
        else
          w[m] = make_float4(in_slot[0], in_slot[CT], in_slot[2 * CT], in_slot[3 * CT]);
      }
      ask(i + kAhead - 1);
      if (r >= depth) continue;
      const float* xr = sm.xs + (r - r0) * TM;
      float xv[TM];
      if constexpr (TM % 4 == 0) {
#pragma unroll
        for (int t = 0; t < TM; t += 4) *(float4*)(xv + t) = *(const float4*)(xr + t);
      } else {
#pragma unroll
        for (int t = 0; t < TM; ++t) xv[t] = xr[t];
      }
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        const uint64_t xx = pack2(xv[t], xv[t]);
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          fma2(acc[t][m][0], xx, pack2(w[m].x, w[m].y));
          fma2(acc[t][m][1], xx, pack2(w[m].z, w[m].w));
        }
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();                    // the ring is free: the sums go there
  // the row groups of a warp, then the warps, each in a fixed order
  float* red = (float*)sm.ring;
  constexpr int L = TM * NM * C;      // of a warp
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 pair = unpack2(acc[t][m][j / 2]);
        float v = j % 2 ? pair.y : pair.x;
#pragma unroll
        for (int o = CT; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane < CT) red[warp * L + (t * NM + m) * C + tile_col<CT, WIDE>(ct, j)] = v;
      }
  __syncthreads();
  for (int e = tid; e < TM * C; e += kThreads) {
    const int t = e / C, c = e - t * C;
    if (t0 + t < cnt && c0 + c < cols) {
      float v[NM];
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        v[m] = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[m] += red[q * L + (t * NM + m) * C + c];
      }
      put(t0 + t, c0 + c, v);
    }
  }
  __syncthreads();
}
template <int CT, bool WIDE, bool POLL, int NM, class In, class Put>
__device__ __forceinline__ void tile(const Args& a, Patience& patience, Smem& sm, const float* const (&W)[NM], int depth,
                                     int cols, int c0, int t0, int cnt, In in, Put put) {
  const int left = cnt - t0;
  if (left == 1)
    tile_tokens<CT, WIDE, POLL, NM, 1>(a, patience, sm, W, depth, cols, c0, t0, cnt, in, put);
  else if (left <= 4)
    tile_tokens<CT, WIDE, POLL, NM, 4>(a, patience, sm, W, depth, cols, c0, t0, cnt, in, put);
  else
    tile_tokens<CT, WIDE, POLL, NM, 8>(a, patience, sm, W, depth, cols, c0, t0, cnt, in, put);
}

template <int CT, int CTD, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2)
decode_experts_kernel(const Args a, const RouteCut cut) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  constexpr int C = 4 * CT, CD = 4 * CTD;
  const int tid = threadIdx.x;
  const float* x = (const float*)a.x;
  float* act = (float*)a.act;
  // tickets start at zero (the previous call's last block left them so), so the
  // first one can be taken while the router still runs
  if (tid == 0) sm.ticket = atomicAdd(a.queue, 1);
  clear_plan(sm.plan, kThreads);
  pdl_wait();
  if (cut.here) {
    pick_all(a, cut, sm.plan, sm.pick, (float*)sm.ring);
    build_plan(sm.plan, nullptr, a.N, a.K, a.E, kThreads);    // ends with a barrier: the ring is free
  } else {
    build_plan(sm.plan, a.top, a.N, a.K, a.E, kThreads);
  }
  const int slots = sm.plan.slots;
  if (tid < 32) {                    // eight slots a lane
    int own[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int u = tid * 8 + i;
      own[i] = sum;
      if (u < slots) sum += (sm.plan.off[u + 1] - sm.plan.off[u] + kTokens - 1) / kTokens;
    }
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, before, o);
      if (tid >= o) before += v;
    }
    before -= sum;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (tid * 8 + i <= slots) sm.chunk0[tid * 8 + i] = before + own[i];
    if (tid == 31 && slots == kMaxExperts) sm.chunk0[slots] = before + sum;
  }
  __syncthreads();
  const int chunks = sm.chunk0[slots];
  const int nft = (int)cdiv(a.F, C), nht = (int)cdiv(a.H, CD);
  const int n_up = chunks * nft, n_down = chunks * nht;
  Patience patience;
  for (;;) {
    int t = sm.ticket;
    __syncthreads();
    if (t >= n_up + n_down) break;
    int next = 0;
    if (tid == 0) next = atomicAdd(a.queue, 1);      // arrives during this tile
    const bool up = t < n_up;
    if (!up) t -= n_up;
    // a slot's tiles in turn, the token chunks of a tile next to one another: they share its weights in L2
    const int tiles = up ? nft : nht;
    int u = 0;
    for (int hi = slots; hi - u > 1;) {
      const int mid = (u + hi) >> 1;
      if (sm.chunk0[mid] * tiles <= t) u = mid; else hi = mid;
    }
    t -= sm.chunk0[u] * tiles;
    const int nch = sm.chunk0[u + 1] - sm.chunk0[u];
    const int c0 = t / nch * (up ? C : CD), t0 = t % nch * kTokens;
    const int e = sm.plan.expert[u], base = sm.plan.off[u], cnt = sm.plan.off[u + 1] - base;
    const size_t eo = (size_t)e * a.H * a.F;
    if (up) {
      if (tid < a.N && ((sm.plan.mask[e][tid >> 5] >> (tid & 31)) & 1u))
        sm.tokens[plan_row(sm.plan, tid, e) - base] = tid;
      const float* const W[2] = {(const float*)a.W1 + eo, (const float*)a.W3 + eo};
      tile<CT, WIDE, false, 2>(
          a, patience, sm, W, a.H, a.F, c0, t0, cnt, [&](int r) { return x + (size_t)sm.tokens[r] * a.H; },
          [&](int r, int c, const float (&v)[2]) { st_word(act + (size_t)(base + r) * a.F + c, silu_f(v[0]) * v[1]); });
    } else {
      const float* const W[1] = {(const float*)a.W2 + eo};
      tile<CTD, true, true, 1>(
          a, patience, sm, W, a.F, a.H, c0, t0, cnt, [&](int r) { return act + (size_t)(base + r) * a.F; },
          [&](int r, int c, const float (&v)[1]) { st_word(a.out + (size_t)(base + r) * a.H + c, v[0]); });
    }
    if (tid == 0) sm.ticket = next;
    __syncthreads();
  }
  // y[n] = sum_k w[n,k] out[row(n,k)], k in order; a static share, nothing waits for it
  const Share sh = share_of(a, (int)gridDim.x);
  for (int at = sh.v0 + tid; at < sh.v1; at += kThreads) {
    const int n = at / sh.per_row, h = (at - n * sh.per_row) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < a.K; k0 += 4) {            // four experts in flight
      float4 v[4];
      const float* o[4];
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + i;
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        w[i] = 0.f;
        if (k < a.K) {
          const int e = cut.here ? sm.pick.id[n][k] : __ldcg(a.top + (size_t)n * a.K + k);
          w[i] = cut.here ? sm.pick.w[n][k] : __ldcg(a.weights + (size_t)n * a.K + k);
          o[i] = a.out + (size_t)plan_row(sm.plan, n, e) * a.H + h;
          v[i] = ld_words4(o[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (k0 + i >= a.K) break;
        while (empty(v[i]) && patience.again(a.cnt, a.status)) v[i] = ld_words4(o[i]);
        s.x = fmaf(w[i], v[i].x, s.x); s.y = fmaf(w[i], v[i].y, s.y);
        s.z = fmaf(w[i], v[i].z, s.z); s.w = fmaf(w[i], v[i].w, s.w);
      }
    }
    *(float4*)((float*)a.y + (size_t)n * a.H + h) = s;
  }
  if (tid == 0 && atomicAdd(a.queue + 1, 1) == (int)gridDim.x - 1) {   // the last block out: ready for the next call
    a.queue[0] = 0;
    a.queue[1] = 0;
  }
}

// ---- host ------------------------------------------------------------------
inline bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline size_t al256(size_t b) { return (b + 255) & ~(size_t)255; }

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
  c.groups = N > 0 ? (int)cdiv(N, c.TG) : 1;
  const int most = (int)cdiv(H, 64), want = (int)cdiv(296, c.groups);
  c.S = most < want ? most : want;
  c.here = N <= kPickTokens && N * c.S * c.EP <= kPickFloats;
  return c;
}

// Room for the cut of any token count up to N: groups * S * TG rows of EP, and
// groups * S < 296 + groups, groups * TG < N + TG, S <= ceil(H / 64).
size_t part_bytes(int N, int H, int E) {
  const int64_t few = round_up(N, 4) * cdiv(H, 64), most = 4 * 296 + N + 4;
  return (size_t)(few < most ? few : most) * route_cut(N, H, E).EP * sizeof(float);
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
  const size_t fill0 = off;
  void* act = take((size_t)N * K * F * sizeof(float));       // or two bf16 numbers each
  void* out = take((size_t)N * K * H * sizeof(float));
  void* pu = dt == MOE_BF16 ? take(umma_up_bytes(N, H, E, K, F)) : nullptr;
  void* pd = dt == MOE_BF16 ? take(umma_down_bytes(N, H, E, K, F)) : nullptr;
  if (a) {
    a->status = (int*)base;
    a->arrive = (int*)(base + 64);
    a->queue = (int*)(base + 192);
    a->cnt = (Counters*)cnt;
    a->zero_ints = (int)(zero / sizeof(int));
    if (dt == MOE_F32 || N <= kDirectTokens) {
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
  // blocks for the filling, where the slices leave SMs free
  const int fillers = a.fill_vecs > 0 && c.S * c.groups < kBlocks ? kBlocks / c.groups - c.S : 0;
  const dim3 grid(c.S + fillers, c.groups);
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

template <int CT, int CTD, bool WIDE>
moe_status experts(const Args& a, const RouteCut& cut, cudaStream_t s) {
  static bool set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    if (cudaFuncSetAttribute(decode_experts_kernel<CT, CTD, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(Smem)) != cudaSuccess) {
      (void)cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  cudaError_t err = cudaSuccess;
  MOE_TRACED("decode_experts", s, (err = launch_after(decode_experts_kernel<CT, CTD, WIDE>, 2 * kBlocks, kThreads, sizeof(Smem),
                                                      s, a, cut)));
  if (err != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}
template <int CT, int CTD>
moe_status experts_at(const Args& a, const RouteCut& cut, bool wide, cudaStream_t s) {
  return wide ? experts<CT, CTD, true>(a, cut, s) : experts<CT, CTD, false>(a, cut, s);
}
moe_status experts_any(const Args& a, const RouteCut& cut, cudaStream_t s) {
  // Tiles of 64 columns where they keep the blocks busy, else narrower ones: each stages
  // its tokens anew and has its start and end to itself.  Up has 32 and 16 columns, down,
  // whose tiles need the least, 16.  13 tokens on 36 experts of 1884/186: down 64 wide
  // 59 us, 32 64, 16 77; one token on two of 1024/1024: 24, 20, 18.  Gate and up of the
  // former 64 wide 59 us, 32 57; of 32 tokens on 16 experts of 1024/1001 96 and 90.
  const double pairs = (double)a.N * a.K;
  const double used = a.E * (1.0 - pow(1.0 - (double)a.K / a.E, a.N));     // experts, of a routing without a bias
  const double chunks = used > pairs / kTokens ? used : pairs / kTokens;
  const int ct = chunks * cdiv(a.F, 64) >= 2 * kBlocks ? 16 : (chunks * cdiv(a.F, 32) >= 2 * kBlocks ? 8 : 4);
  const bool wide = a.F % 4 == 0;
  if (chunks * cdiv(a.H, 64) >= kBlocks)
    return ct == 16 ? experts_at<16, 16>(a, cut, wide, s)
                    : ct == 8 ? experts_at<8, 16>(a, cut, wide, s) : experts_at<4, 16>(a, cut, wide, s);
  return ct == 16 ? experts_at<16, 4>(a, cut, wide, s)
                  : ct == 8 ? experts_at<8, 4>(a, cut, wide, s) : experts_at<4, 4>(a, cut, wide, s);
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
    const moe_status rs = route_any<float>(a, c, !c.here, s);
    return rs != MOE_OK ? rs : experts_any(a, c, s);
  }
  const moe_status rs = route_any<__nv_bfloat16>(a, c, !c.here, s);
  return rs != MOE_OK ? rs : experts_umma(a, c, w.part_up, w.part_down, w.tile_cnt, s);
}

}  // extern "C"
