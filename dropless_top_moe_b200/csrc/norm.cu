// Residual addition and root-mean-square norm in front of the router, forward
// and backward (rows of H, one learned weight per column):
//   forward    h = round(x + r)   (r may be absent: h = x),
//              s = 1 / sqrt(mean_j h_j^2 + eps),  y = h * s * w
//   backward   g = dy * w,  dx = s * g - h * s^3 * mean_j(g_j h_j) + dh,
//              dw_j = sum_n dy_nj * h_nj * s_n
// h is the residual stream as it is kept, rounded to the element type, and y
// is the norm of that rounded h: the backward pass reads h, so it
// differentiates exactly the function the forward computed.  Everything else
// stays in fp32 and is rounded once, at the store.
//
// Both directions do a few operations per byte, so HBM bounds them: four
// elements of N * H moved either way.  A block owns one row at a time and keeps it in
// registers (16-byte loads, VPT vectors a thread), so each element is read
// once; the next row's loads are issued before this row's reduction, which
// keeps loads in flight across the barrier.  The backward accumulates its rows' dw in
// registers; each block then writes one partial row and a second kernel sums the
// partials in block order, so dw has the same bits on every run.
#include "common.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kNormSms = 148;      // blocks are a multiple of this (fixed: dw must not depend on the GPU)
constexpr int kNormMaxVec = 512 * 4;   // 16-byte vectors of a row: 512 threads, 4 each
constexpr int kDwCols = 32, kDwRows = 16;   // block of the dw reduction

// Streamed once: not kept in L1.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

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

template <typename T, int VPT, bool RES>
__global__ void __launch_bounds__(512)
add_rms_norm_kernel(const T* x, const T* residual, const T* __restrict__ weight, int N, int H, float eps,
                    T* h, T* y) {
  constexpr int V = Vec<T>::N;
  __shared__ float red[2][32];
  const int nv = H / V;
  uint4 w[VPT], a[VPT], b[VPT];
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto load = [&](int n) {
    const size_t row = (size_t)n * H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      a[i] = b[i] = zero;
      if (n < N && c < nv) {
        a[i] = ld_stream(x + row + (size_t)c * V);
        if (RES) b[i] = ld_stream(residual + row + (size_t)c * V);
      }
    }
  };
  load(blockIdx.x);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    w[i] = c < nv ? ld_nc_v4(weight + (size_t)c * V) : zero;
  }
  int buf = 0;
  for (int n = blockIdx.x, next; n < N; n = next) {
    next = n < N - (int)gridDim.x ? n + (int)gridDim.x : N;
    const size_t row = (size_t)n * H;
    uint4 hv[VPT];
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[V];
      hv[i] = a[i];
      Vec<T>::to_float(a[i], f);
      if (RES) {
        float g[V];
        Vec<T>::to_float(b[i], g);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] += g[j];
        hv[i] = Vec<T>::from_float(f);      // the residual stream is kept in T
        Vec<T>::to_float(hv[i], f);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) ss[0] = fmaf(f[j], f[j], ss[0]);
    }
    load(next);
    block_sum<1>(ss, red[buf]);
    buf ^= 1;
    const float s = 1.0f / sqrtf(ss[0] / (float)H + eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c >= nv) continue;
      float f[V], g[V];
      Vec<T>::to_float(hv[i], f);
      Vec<T>::to_float(w[i], g);
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = f[j] * s * g[j];
      if (RES) st_v4(h + row + (size_t)c * V, hv[i]);
      st_v4(y + row + (size_t)c * V, Vec<T>::from_float(f));
    }
  }
}

template <typename T, int VPT, bool DH>
__global__ void __launch_bounds__(512, 1)
add_rms_norm_bwd_kernel(const T* dy, const T* h, const T* __restrict__ weight, const T* dh, int N, int H,
                        float eps, T* dx, float* __restrict__ dw_part, T* __restrict__ dw) {
  constexpr int V = Vec<T>::N;
  __shared__ float red[2][64];
  const int nv = H / V;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 w[VPT], a[VPT], b[VPT], d[VPT];
  float acc[VPT][V];
  auto load = [&](int n) {
    const size_t row = (size_t)n * H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      a[i] = b[i] = d[i] = zero;
      if (n < N && c < nv) {
        a[i] = ld_stream(h + row + (size_t)c * V);
        b[i] = ld_stream(dy + row + (size_t)c * V);
        if (DH) d[i] = ld_stream(dh + row + (size_t)c * V);
      }
    }
  };
  constexpr bool kAhead = VPT < 4;     // four vectors of three rows leave no registers for the next row's
  if (kAhead) load(blockIdx.x);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    w[i] = c < nv ? ld_nc_v4(weight + (size_t)c * V) : zero;
#pragma unroll
    for (int j = 0; j < V; ++j) acc[i][j] = 0.f;
  }
  int buf = 0;
  for (int n = blockIdx.x, next; n < N; n = next) {
    next = n < N - (int)gridDim.x ? n + (int)gridDim.x : N;
    const size_t row = (size_t)n * H;
    uint4 hv[VPT], gv[VPT], dv[VPT];
    if (!kAhead) load(n);
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      hv[i] = a[i];
      gv[i] = b[i];
      dv[i] = d[i];
      float f[V], g[V], wf[V];
      Vec<T>::to_float(hv[i], f);
      Vec<T>::to_float(gv[i], g);
      Vec<T>::to_float(w[i], wf);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sum[0] = fmaf(f[j], f[j], sum[0]);
        sum[1] = fmaf(g[j] * wf[j], f[j], sum[1]);
      }
    }
    if (kAhead) load(next);
    block_sum<2>(sum, red[buf]);
    buf ^= 1;
    const float s = 1.0f / sqrtf(sum[0] / (float)H + eps);
    const float m = sum[1] / (float)H * s;       // mean(g * xhat)
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c >= nv) continue;
      float f[V], g[V], wf[V], r[V];
      Vec<T>::to_float(hv[i], f);
      Vec<T>::to_float(gv[i], g);
      Vec<T>::to_float(w[i], wf);
      Vec<T>::to_float(dv[i], r);
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

// dw[c] = sum over the blocks' partial rows: kDwRows strided sums, then those
// in order.
template <typename T>
__global__ void __launch_bounds__(kDwCols * kDwRows)
rms_norm_dw_kernel(const float* __restrict__ part, int G, int H, T* __restrict__ dw) {
  __shared__ float red[kDwRows][kDwCols];
  const int tc = threadIdx.x % kDwCols, tr = threadIdx.x / kDwCols;
  const int c = blockIdx.x * kDwCols + tc;
  float s = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int g = tr; g < G; g += kDwRows) s += part[(size_t)g * H + c];
  }
  red[tr][tc] = s;
  __syncthreads();
  if (tr == 0 && c < H) {
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < kDwRows; ++r) t += red[r][tc];
    dw[c] = from_f<T>(t);
  }
}

// Threads of a row's block and vectors a thread: the fewest vectors (1, 2, 4)
// that keep the block within `cap` threads.
struct NormShape {
  int threads, vpt;
};
NormShape norm_shape(int nv, int cap) {
  NormShape s;
  s.vpt = 1;
  while (s.vpt < 4 && nv > cap * s.vpt) s.vpt *= 2;
  s.threads = (int)round_up(cdiv(nv, s.vpt), 32);
  return s;
}

int norm_blocks(int N, int threads, int most_threads) {
  int per_sm = most_threads / threads;
  if (per_sm < 1) per_sm = 1;
  if (per_sm > 16) per_sm = 16;
  const int64_t g = (int64_t)kNormSms * per_sm;
  return (int)(N < g ? N : g);
}

constexpr int kFwdCap = 256, kFwdThreads = 1024;   // threads of a block before rows take more vectors; of an SM
constexpr int kBwdCap = 256, kBwdThreads = 512;

moe_status norm_check(int N, int H, moe_dtype dt) {
  if (dt != MOE_F32 && dt != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (N < 0 || H <= 0) return MOE_ERR_INVALID_ARG;
  const int V = dt == MOE_F32 ? 4 : 8;
  if (H % V) return MOE_ERR_UNSUPPORTED;
  if (H / V > kNormMaxVec) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

NormShape shape_of(int H, moe_dtype dt, int cap) {
  const int nv = H / (dt == MOE_F32 ? 4 : 8);
  return norm_shape(nv, nv > cap * 2 ? 512 : cap);
}

size_t bwd_partials(int N, int H, moe_dtype dt) {
  const int G = norm_blocks(N, shape_of(H, dt, kBwdCap).threads, kBwdThreads);
  return G > 1 ? (size_t)G * H * sizeof(float) : 0;
}

template <typename T, int VPT>
void launch_fwd(const void* x, const void* r, const void* w, int N, int H, float eps, void* h, void* y,
                int blocks, int threads, cudaStream_t s) {
  if (r)
    MOE_TRACED("add_rms_norm", s, (add_rms_norm_kernel<T, VPT, true><<<blocks, threads, 0, s>>>(
                                      (const T*)x, (const T*)r, (const T*)w, N, H, eps, (T*)h, (T*)y)));
  else
    MOE_TRACED("rms_norm", s, (add_rms_norm_kernel<T, VPT, false><<<blocks, threads, 0, s>>>(
                                  (const T*)x, nullptr, (const T*)w, N, H, eps, nullptr, (T*)y)));
}

template <typename T, int VPT>
void launch_bwd(const void* dy, const void* h, const void* w, const void* dh, int N, int H, float eps, void* dx,
                float* part, void* dw, int blocks, int threads, cudaStream_t s) {
  if (dh)
    MOE_TRACED("add_rms_norm_bwd", s, (add_rms_norm_bwd_kernel<T, VPT, true><<<blocks, threads, 0, s>>>(
                                          (const T*)dy, (const T*)h, (const T*)w, (const T*)dh, N, H, eps, (T*)dx,
                                          part, (T*)dw)));
  else
    MOE_TRACED("rms_norm_bwd", s, (add_rms_norm_bwd_kernel<T, VPT, false><<<blocks, threads, 0, s>>>(
                                      (const T*)dy, (const T*)h, (const T*)w, nullptr, N, H, eps, (T*)dx, part,
                                      (T*)dw)));
}

template <typename T>
moe_status norm_fwd(const void* x, const void* r, const void* w, int N, int H, moe_dtype dt, float eps, void* h,
                    void* y, cudaStream_t s) {
  const NormShape sh = shape_of(H, dt, kFwdCap);
  const int blocks = norm_blocks(N, sh.threads, kFwdThreads);
  if (sh.vpt == 1) launch_fwd<T, 1>(x, r, w, N, H, eps, h, y, blocks, sh.threads, s);
  else if (sh.vpt == 2) launch_fwd<T, 2>(x, r, w, N, H, eps, h, y, blocks, sh.threads, s);
  else launch_fwd<T, 4>(x, r, w, N, H, eps, h, y, blocks, sh.threads, s);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

template <typename T>
moe_status norm_bwd(const void* dy, const void* h, const void* w, const void* dh, int N, int H, moe_dtype dt,
                    float eps, void* dx, void* dw, float* part, cudaStream_t s) {
  const NormShape sh = shape_of(H, dt, kBwdCap);
  const int blocks = norm_blocks(N, sh.threads, kBwdThreads);
  if (sh.vpt == 1) launch_bwd<T, 1>(dy, h, w, dh, N, H, eps, dx, part, dw, blocks, sh.threads, s);
  else if (sh.vpt == 2) launch_bwd<T, 2>(dy, h, w, dh, N, H, eps, dx, part, dw, blocks, sh.threads, s);
  else launch_bwd<T, 4>(dy, h, w, dh, N, H, eps, dx, part, dw, blocks, sh.threads, s);
  MOE_LAUNCH_CHECK();
  if (blocks > 1) {
    MOE_TRACED("rms_norm_dw", s, (rms_norm_dw_kernel<T><<<(unsigned)cdiv(H, kDwCols), kDwCols * kDwRows, 0, s>>>(
                                     part, blocks, H, (T*)dw)));
    MOE_LAUNCH_CHECK();
  }
  return MOE_OK;
}

inline bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Two buffers that share memory without being the same one: a row's block
// would overwrite rows that others still have to read.
bool cross(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || (a == b && na == nb)) return false;
  return (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

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
  if (h == y || cross(h, all, y, all) || cross(h, all, weight, row) || cross(y, all, weight, row) ||
      cross(h, all, x, all) || cross(h, all, residual, all) || cross(y, all, x, all) || cross(y, all, residual, all))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  return dt == MOE_F32 ? norm_fwd<float>(x, residual, weight, N, H, dt, eps, h, y, s)
                       : norm_fwd<__nv_bfloat16>(x, residual, weight, N, H, dt, eps, h, y, s);
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
  if (N > 0 && (cross(dx, all, dy, all) || cross(dx, all, h, all) || cross(dx, all, dh, all) ||
                cross(dx, all, weight, row) || cross(dx, all, dweight, row) || cross(dweight, row, dy, all) ||
                cross(dweight, row, h, all) || cross(dweight, row, dh, all) || dweight == weight ||
                cross(dweight, row, weight, row)))
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
  return dt == MOE_F32 ? norm_bwd<float>(dy, h, weight, dh, N, H, dt, eps, dx, dweight, part, s)
                       : norm_bwd<__nv_bfloat16>(dy, h, weight, dh, N, H, dt, eps, dx, dweight, part, s);
}

}  // extern "C"
