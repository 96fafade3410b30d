// Residual addition and root-mean-square norm in front of the router, forward
// and backward (rows of H, one learned weight per column):
//   forward    h = round(x + r)   (r may be absent: h = x),
//              s = 1 / sqrt(mean_j h_j^2 + eps),  y = h * s * w
//   backward   g = dy * w,  dx = s * g - h * s^3 * mean_j(g_j h_j) + dh  (dh may be absent),
//              dw_j = sum_n dy_nj * h_nj * s_n
// h is the residual stream as it is kept, rounded to the element type, and y
// is the norm of that rounded h: the backward pass reads h, so it
// differentiates exactly the function the forward computed.  Everything else
// stays in fp32 and is rounded once, at the store.
//
// Both directions do a few operations per byte, so HBM bounds them: four
// elements of N * H moved either way.  A block owns one row at a time, holds it in
// registers (VPT 16-byte vectors a thread) and so reads each element once.  The rows to
// come are on their way meanwhile: every thread copies its own vectors of the next
// rows to shared memory (cp.async), one or two rows ahead, and reads only what it
// copied itself, so this costs neither registers nor barriers; one barrier a row
// remains, in the row's sum.  The backward accumulates its rows' dw in registers; each
// block then writes one partial row and a second kernel sums the partials in
// block order, so dw has the same bits on every run.
#include <string.h>

#include "common.cuh"
#include "kernels.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kNormSms = 148;      // blocks are a multiple of this (fixed: dw must not depend on the GPU)
constexpr int kNormMaxVec = 512 * 4;   // 16-byte vectors of a row: 512 threads, 4 each
constexpr int kDwCols = 8, kDwRows = 64;    // block of the dw reduction: 32-byte columns, many rows in flight

__device__ __forceinline__ void copy16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// This thread's vectors of the rows to come: each of D slots holds NIN operands' VPT vectors.
template <typename T, int VPT, int NIN, int D>
struct Rows {
  const T* src[NIN];
  uint4* mine;        // [slot][operand][vector][thread]
  int N, H, nv, slot;
  __device__ __forceinline__ uint4* at(int s, int o, int i) const {
    return mine + ((s * NIN + o) * VPT + i) * blockDim.x;
  }
  __device__ __forceinline__ void ask(int s, int n) {
    if (n < N) {
#pragma unroll
      for (int o = 0; o < NIN; ++o)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = threadIdx.x + i * blockDim.x;
          if (c < nv) copy16(at(s, o, i), src[o] + (size_t)n * H + (size_t)c * Vec<T>::N);
        }
    }
    copy_commit();      // an empty group past the last row keeps the count
  }
  __device__ __forceinline__ static int after(int n, int N) {
    return n < N - (int)gridDim.x ? n + (int)gridDim.x : N;
  }
  // The first D - 1 rows; returns the row after them.
  __device__ __forceinline__ int begin(int n) {
#pragma unroll
    for (int s = 0; s < D - 1; ++s) {
      ask(s, n);
      if (n < N) n = after(n, N);
    }
    slot = 0;
    return n;
  }
  // The current row's vectors, and row `ahead` asked for into the slot read last.
  __device__ __forceinline__ void take(int ahead, uint4 (&v)[NIN][VPT]) {
    // the oldest of D - 1 groups has arrived
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 2) : "memory");
    ask(slot == 0 ? D - 1 : slot - 1, ahead);
#pragma unroll
    for (int o = 0; o < NIN; ++o)
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        v[o][i] = c < nv ? *at(slot, o, i) : make_uint4(0, 0, 0, 0);
      }
    slot = slot == D - 1 ? 0 : slot + 1;
  }
};

// Sum of NV values a thread over the block, in a fixed order, on every thread.
// `red` alternates between two buffers from call to call: one barrier a call.
template <int NV>
__device__ __forceinline__ void block_sum(float (&v)[NV], float* red) {
  const int nw = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = warp_sum(v[i]);
  if (nw == 1) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) red[i * 32 + warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = warp_sum(lane < nw ? red[i * 32 + lane] : 0.f);
}

template <typename T, int VPT, int D, bool RES>
__global__ void __launch_bounds__(512)
add_rms_norm_kernel(const T* x, const T* residual, const T* __restrict__ weight, int N, int H, float eps,
                    T* h, T* y) {
  constexpr int V = Vec<T>::N, NIN = RES ? 2 : 1;
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float red[2][32];
  const int nv = H / V;
  Rows<T, VPT, NIN, D> rows;
  rows.src[0] = x;
  if constexpr (RES) rows.src[1] = residual;
  rows.mine = ring + threadIdx.x;
  rows.N = N; rows.H = H; rows.nv = nv;
  int ahead = rows.begin(blockIdx.x);
  uint4 w[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    w[i] = c < nv ? ld_nc_v4(weight + (size_t)c * V) : make_uint4(0, 0, 0, 0);
  }
  int buf = 0;
  for (int n = blockIdx.x, next; n < N; n = next) {
    next = rows.after(n, N);
    const size_t row = (size_t)n * H;
    uint4 v[NIN][VPT];
    rows.take(ahead, v);
    if (ahead < N) ahead = rows.after(ahead, N);
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[V];
      Vec<T>::to_float(v[0][i], f);
      if constexpr (RES) {
        float g[V];
        Vec<T>::to_float(v[1][i], g);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] += g[j];
        v[0][i] = Vec<T>::from_float(f);      // the residual stream is kept in T
        Vec<T>::to_float(v[0][i], f);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) ss[0] = fmaf(f[j], f[j], ss[0]);
    }
    block_sum<1>(ss, red[buf]);
    buf ^= 1;
    const float s = 1.0f / sqrtf(ss[0] / (float)H + eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c >= nv) continue;
      float f[V], g[V];
      Vec<T>::to_float(v[0][i], f);
      Vec<T>::to_float(w[i], g);
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = f[j] * s * g[j];
      if (RES) st_v4(h + row + (size_t)c * V, v[0][i]);
      st_v4(y + row + (size_t)c * V, Vec<T>::from_float(f));
    }
  }
}

template <typename T, int VPT, int D, bool DH>
__global__ void __launch_bounds__(512)
add_rms_norm_bwd_kernel(const T* dy, const T* h, const T* __restrict__ weight, const T* dh, int N, int H,
                        float eps, T* dx, float* __restrict__ dw_part, T* __restrict__ dw) {
  constexpr int V = Vec<T>::N, NIN = DH ? 3 : 2;
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float red[2][64];
  pdl_launch();
  const int nv = H / V;
  Rows<T, VPT, NIN, D> rows;
  rows.src[0] = h;
  rows.src[1] = dy;
  if constexpr (DH) rows.src[2] = dh;
  rows.mine = ring + threadIdx.x;
  rows.N = N; rows.H = H; rows.nv = nv;
  int ahead = rows.begin(blockIdx.x);
  uint4 w[VPT];
  float acc[VPT][V];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    w[i] = c < nv ? ld_nc_v4(weight + (size_t)c * V) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < V; ++j) acc[i][j] = 0.f;
  }
  int buf = 0;
  for (int n = blockIdx.x, next; n < N; n = next) {
    next = rows.after(n, N);
    const size_t row = (size_t)n * H;
    uint4 v[NIN][VPT];
    rows.take(ahead, v);
    if (ahead < N) ahead = rows.after(ahead, N);
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[V], g[V], wf[V];
      Vec<T>::to_float(v[0][i], f);
      Vec<T>::to_float(v[1][i], g);
      Vec<T>::to_float(w[i], wf);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sum[0] = fmaf(f[j], f[j], sum[0]);
        sum[1] = fmaf(g[j] * wf[j], f[j], sum[1]);
      }
    }
    block_sum<2>(sum, red[buf]);
    buf ^= 1;
    const float s = 1.0f / sqrtf(sum[0] / (float)H + eps);
    const float m = sum[1] / (float)H * s;       // mean(g * xhat)
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c >= nv) continue;
      float f[V], g[V], wf[V], r[V];
      Vec<T>::to_float(v[0][i], f);
      Vec<T>::to_float(v[1][i], g);
      Vec<T>::to_float(w[i], wf);
      if constexpr (DH) Vec<T>::to_float(v[2][i], r);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xhat = f[j] * s;
        acc[i][j] = fmaf(g[j], xhat, acc[i][j]);
        const float t = s * (g[j] * wf[j] - xhat * m);
        r[j] = DH ? t + r[j] : t;
      }
      st_v4(dx + row + (size_t)c * V, Vec<T>::from_float(r));
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c >= nv) continue;
    if (gridDim.x == 1) {                         // one block: its sums are dw
      st_v4(dw + (size_t)c * V, Vec<T>::from_float(acc[i]));
    } else {
      float* p = dw_part + (size_t)blockIdx.x * H + (size_t)c * V;
#pragma unroll
      for (int j = 0; j < V; j += 4) *(float4*)(p + j) = make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
    }
  }
}

// dw[c] = sum over the blocks' partial rows: kDwRows strided sums, eight loads of
// each in flight, then those in a fixed order.  The partials are still being written when this
// kernel starts: no restrict and no read-only path for them.
template <typename T>
__global__ void __launch_bounds__(kDwCols * kDwRows)
rms_norm_dw_kernel(const float* part, int G, int H, T* __restrict__ dw) {
  static_assert(kDwCols == 8 && kDwRows % 4 == 0, "four rows of eight columns a warp");
  __shared__ float red[kDwRows / 4][kDwCols];
  const int tc = threadIdx.x % kDwCols, tr = threadIdx.x / kDwCols;
  const int c = blockIdx.x * kDwCols + tc;
  float s = 0.f;
  pdl_wait();
  if (c < H) {
    for (int g = tr; g < G; g += 8 * kDwRows) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = g + i * kDwRows < G ? part[(size_t)(g + i * kDwRows) * H + c] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
  }
  s += __shfl_xor_sync(0xffffffffu, s, 8);
  s += __shfl_xor_sync(0xffffffffu, s, 16);
  if ((threadIdx.x & 31) < kDwCols) red[tr / 4][tc] = s;
  __syncthreads();
  if (tr == 0 && c < H) {
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < kDwRows / 4; ++r) t += red[r][tc];
    dw[c] = from_f<T>(t);
  }
}

// Threads of a row's block, vectors a thread, rows under way, blocks.  Two vectors a
// thread where the row allows; as many blocks an SM as kSmThreads and shared memory
// allow; two rows ahead for the backward and for rows that leave one block an SM, one
// row for the forward's others.  More under way was slower on long rows (16384 x 4096
// bf16: forward 87 us, 95 with two rows ahead, 97 with twice the threads; backward
// 83 us, 87 with one row ahead, 103 with three blocks an SM).
constexpr int kSmThreads = 512, kSmBytes = 220 * 1024;
struct NormShape {
  int threads, vpt, depth, blocks;
  size_t smem;
};
NormShape norm_shape(int N, int H, moe_dtype dt, int nin, bool bwd) {
  const int nv = H / (dt == MOE_F32 ? 4 : 8);
  const int cap = nv > 512 ? 512 : (nv > 256 ? 256 : 128);
  NormShape s;
  s.vpt = 1;
  while (s.vpt < 4 && nv > cap * s.vpt) s.vpt *= 2;
  s.threads = (int)round_up(cdiv(nv, s.vpt), 32);
  int per_sm = kSmThreads / s.threads;
  const size_t row = (size_t)nin * s.vpt * s.threads * 16;
  s.depth = bwd || per_sm == 1 || nv <= 256 ? 3 : 2;
  if (s.depth * row > kSmBytes) s.depth = 2;
  s.smem = s.depth * row;
  if (per_sm * s.smem > kSmBytes) per_sm = (int)(kSmBytes / s.smem);
  const int64_t g = (int64_t)kNormSms * per_sm;
  s.blocks = (int)(N < g ? N : g);
  return s;
}

moe_status norm_check(int N, int H, moe_dtype dt) {
  if (dt != MOE_F32 && dt != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (N < 0 || H <= 0) return MOE_ERR_INVALID_ARG;
  const int V = dt == MOE_F32 ? 4 : 8;
  if (H % V) return MOE_ERR_UNSUPPORTED;
  if (H / V > kNormMaxVec) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t bwd_partials(int N, int H, moe_dtype dt) {
  const int a = norm_shape(N, H, dt, 2, true).blocks, b = norm_shape(N, H, dt, 3, true).blocks;
  const int G = a > b ? a : b;
  return G > 1 ? (size_t)G * H * sizeof(float) : 0;
}

// Once a kernel and device: more shared memory than 48 KB.
template <class Kernel>
bool allow_smem(Kernel k, bool (&set)[64]) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && set[dev]) return true;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmBytes) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  if (dev >= 0 && dev < 64) set[dev] = true;
  return true;
}

template <typename T, int VPT, int D, bool RES>
bool launch_fwd(const void* x, const void* r, const void* w, int N, int H, float eps, void* h, void* y,
                const NormShape& sh, cudaStream_t s) {
  static bool set[64] = {false};
  if (!allow_smem(add_rms_norm_kernel<T, VPT, D, RES>, set)) return false;
  MOE_TRACED(RES ? "add_rms_norm" : "rms_norm", s,
             (add_rms_norm_kernel<T, VPT, D, RES><<<sh.blocks, sh.threads, sh.smem, s>>>(
                 (const T*)x, (const T*)r, (const T*)w, N, H, eps, (T*)h, (T*)y)));
  return true;
}
template <typename T, int VPT, int D, bool DH>
bool launch_bwd(const void* dy, const void* h, const void* w, const void* dh, int N, int H, float eps, void* dx,
                float* part, void* dw, const NormShape& sh, cudaStream_t s) {
  static bool set[64] = {false};
  if (!allow_smem(add_rms_norm_bwd_kernel<T, VPT, D, DH>, set)) return false;
  MOE_TRACED(DH ? "add_rms_norm_bwd" : "rms_norm_bwd", s,
             (add_rms_norm_bwd_kernel<T, VPT, D, DH><<<sh.blocks, sh.threads, sh.smem, s>>>(
                 (const T*)dy, (const T*)h, (const T*)w, (const T*)dh, N, H, eps, (T*)dx, part, (T*)dw)));
  return true;
}

template <typename T, bool RES>
moe_status norm_fwd(const void* x, const void* r, const void* w, int N, int H, moe_dtype dt, float eps, void* h,
                    void* y, cudaStream_t s) {
  const NormShape sh = norm_shape(N, H, dt, RES ? 2 : 1, false);
  const bool deep = sh.depth == 3;
#define MOE_NORM_FWD(VPT) (deep ? launch_fwd<T, VPT, 3, RES>(x, r, w, N, H, eps, h, y, sh, s) \
                                : launch_fwd<T, VPT, 2, RES>(x, r, w, N, H, eps, h, y, sh, s))
  const bool ok = sh.vpt == 1 ? MOE_NORM_FWD(1) : sh.vpt == 2 ? MOE_NORM_FWD(2) : MOE_NORM_FWD(4);
#undef MOE_NORM_FWD
  if (!ok) return MOE_ERR_CUDA;
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

template <typename T, bool DH>
moe_status norm_bwd(const void* dy, const void* h, const void* w, const void* dh, int N, int H, moe_dtype dt,
                    float eps, void* dx, void* dw, float* part, cudaStream_t s) {
  const NormShape sh = norm_shape(N, H, dt, DH ? 3 : 2, true);
  const bool deep = sh.depth == 3;
#define MOE_NORM_BWD(VPT) (deep ? launch_bwd<T, VPT, 3, DH>(dy, h, w, dh, N, H, eps, dx, part, dw, sh, s) \
                                : launch_bwd<T, VPT, 2, DH>(dy, h, w, dh, N, H, eps, dx, part, dw, sh, s))
  const bool ok = sh.vpt == 1 ? MOE_NORM_BWD(1) : sh.vpt == 2 ? MOE_NORM_BWD(2) : MOE_NORM_BWD(4);
#undef MOE_NORM_BWD
  if (!ok) return MOE_ERR_CUDA;
  MOE_LAUNCH_CHECK();
  if (sh.blocks > 1) {
    cudaError_t err = cudaSuccess;
    MOE_TRACED("rms_norm_dw", s,
               (err = launch_after(rms_norm_dw_kernel<T>, (unsigned)cdiv(H, kDwCols), kDwCols * kDwRows, 0, s,
                                   (const float*)part, sh.blocks, H, (T*)dw)));
    if (err != cudaSuccess) {
      (void)cudaGetLastError();
      return MOE_ERR_CUDA;
    }
  }
  return MOE_OK;
}

inline bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  return a && b && (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}
// Two [N,H] buffers that share memory without being the same one: a row's block
// would overwrite rows that others still have to read.
bool cross(const void* a, const void* b, size_t n) { return a != b && overlap(a, n, b, n); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_add_rms_norm(const void* x, const void* residual, const void* weight, int32_t N, int32_t H,
                            moe_dtype dt, float eps, void* h, void* y, moe_stream_t stream) {
  const moe_status st = norm_check(N, H, dt);
  if (st != MOE_OK) return st;
  if (!(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (!weight || (N > 0 && (!x || !y || (residual && !h)))) return MOE_ERR_INVALID_ARG;
  if (!al16(x) || !al16(residual) || !al16(weight) || !al16(h) || !al16(y)) return MOE_ERR_INVALID_ARG;
  if (N == 0) return MOE_OK;
  if (!residual) h = nullptr;
  const size_t row = (size_t)H * (dt == MOE_F32 ? 4 : 2), all = row * N;
  if (overlap(h, all, y, all) || overlap(h, all, weight, row) || overlap(y, all, weight, row) ||
      cross(h, x, all) || cross(h, residual, all) || cross(y, x, all) || cross(y, residual, all))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (dt == MOE_F32)
    return residual ? norm_fwd<float, true>(x, residual, weight, N, H, dt, eps, h, y, s)
                    : norm_fwd<float, false>(x, nullptr, weight, N, H, dt, eps, nullptr, y, s);
  return residual ? norm_fwd<__nv_bfloat16, true>(x, residual, weight, N, H, dt, eps, h, y, s)
                  : norm_fwd<__nv_bfloat16, false>(x, nullptr, weight, N, H, dt, eps, nullptr, y, s);
}

size_t moe_add_rms_norm_bwd_workspace_size(int32_t N, int32_t H, moe_dtype dt) {
  if (norm_check(N, H, dt) != MOE_OK) return 0;
  return kStatusBytes + (size_t)round_up((int64_t)bwd_partials(N, H, dt), 256);
}

moe_status moe_add_rms_norm_bwd(const void* dy, const void* h, const void* weight, const void* dh, int32_t N,
                                int32_t H, moe_dtype dt, float eps, void* dx, void* dweight, void* ws,
                                size_t ws_bytes, moe_stream_t stream) {
  const moe_status st = norm_check(N, H, dt);
  if (st != MOE_OK) return st;
  if (!(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (!weight || !dweight || (N > 0 && (!dy || !h || !dx))) return MOE_ERR_INVALID_ARG;
  if (!al16(dy) || !al16(h) || !al16(weight) || !al16(dh) || !al16(dx) || !al16(dweight)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < moe_add_rms_norm_bwd_workspace_size(N, H, dt)) return MOE_ERR_WORKSPACE;
  if (!al16(ws)) return MOE_ERR_INVALID_ARG;
  const size_t row = (size_t)H * (dt == MOE_F32 ? 4 : 2), all = row * N;
  if (overlap(dweight, row, weight, row)) return MOE_ERR_INVALID_ARG;
  if (N > 0 && (cross(dx, dy, all) || cross(dx, h, all) || cross(dx, dh, all) || overlap(dx, all, weight, row) ||
                overlap(dx, all, dweight, row) || overlap(dweight, row, dy, all) || overlap(dweight, row, h, all) ||
                overlap(dweight, row, dh, all)))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (N == 0) {   // no rows: an empty sum
    if (cudaMemsetAsync(dweight, 0, (size_t)H * (dt == MOE_F32 ? 4 : 2), s) != cudaSuccess) {
      (void)cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    return MOE_OK;
  }
  float* part = (float*)((char*)ws + kStatusBytes);
  if (dt == MOE_F32)
    return dh ? norm_bwd<float, true>(dy, h, weight, dh, N, H, dt, eps, dx, dweight, part, s)
              : norm_bwd<float, false>(dy, h, weight, dh, N, H, dt, eps, dx, dweight, part, s);
  return dh ? norm_bwd<__nv_bfloat16, true>(dy, h, weight, dh, N, H, dt, eps, dx, dweight, part, s)
            : norm_bwd<__nv_bfloat16, false>(dy, h, weight, dh, N, H, dt, eps, dx, dweight, part, s);
}

}  // extern "C"
