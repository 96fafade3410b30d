// Global norm of a list of gradients and their scaling:
//   norm = sqrt(sum over every element g^2),
//   out  = round(g * f),  f = min(1, max_norm / (norm + 1e-6)).
// Two launches: one sums the squares into one double a block, the other adds those in
// block order (so the norm, and with it every bit of the scaled gradients, is
// the same on every run and on every rank that holds the same gradients, wherever
// they lie in memory) and scales.  In place with f = 1 there is nothing to write and the second launch
// returns after the sum.
//
// Bound by HBM: two reads and a write of every gradient, less what the second
// pass still finds in L2.  It walks the chunks backwards for that: the first pass
// read the last ones most recently.
//
// The tensors travel in the kernel's parameters (no copy to the device that a
// captured graph would have to keep); a longer list takes several launches.
// A tensor is cut into chunks of kChunkVec vectors of 16 bytes, counted from its first
// element for the sum and from its first 16-byte boundary on for the scaling, where
// the few elements before and after go one by one.
//
// Squares are summed in fp32 over kSumVec vectors, then in double.  An fp32 sum that
// overflowed, or so small that squares may have underflowed, is taken again in
// double, so the norm holds for gradients of any magnitude.
//
// Measured: 3.2 GB of bf16 gradients 1.45 ms (9.7 GB moved: 6.7 TB/s), 288 MB in 60
// tensors 139 to 144 us; 16 KB chunks and two thirds of the blocks took 1.60 ms, 150 us.
#include <float.h>

#include <algorithm>
#include <new>
#include <utility>
#include <vector>

#include "common.cuh"
#include "kernels.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kClipThreads = 256;
constexpr int kChunkPer = 8;                              // vectors a thread takes of a chunk
constexpr int kChunkVec = kClipThreads * kChunkPer;       // 32 KB
constexpr int kSumVec = 4;                                // of them added in fp32 at a time
constexpr int kClipBlocks = 148 * 12;                     // most blocks a launch (fixed: the sum's order)

struct ClipTensor {
  const void* g;
  void* out;
  int64_t numel;
  int32_t first;       // first chunk of this tensor in its launch
  int32_t dt;
};
template <int M>
struct ClipTable {
  ClipTensor t[M];
  int32_t count;
  int32_t chunks;
};
constexpr int kClipMax = 768;    // tensors a launch: 24.6 KB of parameters

template <typename T>
__device__ __forceinline__ int head_of(const T* p, int64_t numel) {
  const int h = (int)(((16u - ((uintptr_t)p & 15u)) & 15u) / sizeof(T));
  return numel < h ? (int)numel : h;
}

// Tensor of chunk c: the last one whose first chunk is <= c.
template <int M>
__device__ __forceinline__ int tensor_of(const ClipTable<M>& tab, int c) {
  int lo = 0, hi = tab.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.t[mid].first <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The sum of squares goes by element index alone: vector i of a tensor is its elements
// V i to V i + V - 1, wherever the tensor starts, so that two ranks that hold the same gradients
// at other offsets from a 16-byte boundary have the same norm to the last bit.  A tensor off the
// boundary pays two loads a vector for it (800 MB: the whole call 422 us for 385 in bf16, 394 for 380 in fp32).

// kSumVec vectors of a thread in fp32, in double where that left the range.
template <typename T>
__device__ __forceinline__ double vec_squares(const uint4* v) {
  constexpr int V = Vec<T>::N;
  float s = 0.f;
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < kSumVec; ++i) {
    float f[V];
    Vec<T>::to_float(v[i], f);
    bits |= v[i].x | v[i].y | v[i].z | v[i].w;
#pragma unroll
    for (int j = 0; j < V; ++j) s = fmaf(f[j], f[j], s);
  }
  if ((s > 1e-30f && s < 1e38f) || bits == 0) return (double)s;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < kSumVec; ++i) {
    float f[V];
    Vec<T>::to_float(v[i], f);
#pragma unroll
    for (int j = 0; j < V; ++j) sum += (double)f[j] * (double)f[j];
  }
  return sum;
}

// A vector of a tensor that starts `off` bytes past a 16-byte boundary, out of the two aligned ones
// that cover it.
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int off) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (off & 8) {
#pragma unroll
    for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
  }
  if (off & 4) {
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
  }
  const int bits = (off & 2) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}
template <typename T>
__device__ __forceinline__ uint4 load_each(const T* p) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(T) == 4) w[j] = __ldg((const uint32_t*)p + j);
    else w[j] = __ldg((const uint16_t*)p + 2 * j) | (uint32_t)__ldg((const uint16_t*)p + 2 * j + 1) << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum of the squares of one thread's part of a chunk.
template <typename T>
__device__ __forceinline__ double chunk_squares(const T* g, int64_t numel, int chunk, bool last) {
  constexpr int V = Vec<T>::N;
  const int64_t nvec = numel / V, left = nvec - (int64_t)chunk * kChunkVec;
  const int n = left < kChunkVec ? (int)left : kChunkVec;       // vectors of this chunk
  const int off = (int)((uintptr_t)g & 15u);
  const char* from = (const char*)g + (int64_t)chunk * kChunkVec * 16;
  const uint4 none = make_uint4(0, 0, 0, 0);
  double sum = 0.0;
  uint4 v[kChunkPer];
  if (off == 0) {
#pragma unroll
    for (int i = 0; i < kChunkPer; ++i) {
      const int at = threadIdx.x + i * kClipThreads;
      v[i] = at < n ? ld_nc_v4(from + (size_t)at * 16) : none;
    }
#pragma unroll
    for (int h = 0; h < kChunkPer; h += kSumVec) sum += vec_squares<T>(v + h);
  } else {
    // A vector lies across two aligned ones, of which the second is in L1 as the next lane's first.  Those of
    // the tensor's first and last vector reach past it: these two go element by element.
    const int head = chunk == 0 ? 0 : -1, tail = left <= kChunkVec ? n - 1 : n;
    const char* base = from - off;
#pragma unroll
    for (int h = 0; h < kChunkPer; h += kSumVec) {
      uint4 o[kSumVec];
#pragma unroll
      for (int i = 0; i < kSumVec; ++i) {
        const int at = threadIdx.x + (h + i) * kClipThreads;
        const bool in = at < tail && at != head;
        v[i] = in ? ld_nc_v4(base + (size_t)at * 16) : none;
        o[i] = in ? ld_nc_v4(base + (size_t)at * 16 + 16) : none;
      }
#pragma unroll
      for (int i = 0; i < kSumVec; ++i) {
        const int at = threadIdx.x + (h + i) * kClipThreads;
        v[i] = shifted(v[i], o[i], off);
        if (at < n && (at >= tail || at == head)) v[i] = load_each(g + ((int64_t)chunk * kChunkVec + at) * V);
      }
      sum += vec_squares<T>(v);
    }
  }
  if (last) {                            // the elements after the last whole vector
    const int64_t at = nvec * V + threadIdx.x;
    if (at < numel) {
      const double d = (double)to_f<T>(g[at]);
      sum += d * d;
    }
  }
  return sum;
}

__device__ __forceinline__ double block_sum_f64(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kClipThreads / 32; ++w) s += red[w];
  return s;
}

template <int M>
__global__ void __launch_bounds__(kClipThreads)
grad_squares_kernel(const __grid_constant__ ClipTable<M> tab, double* __restrict__ part) {
  __shared__ double red[kClipThreads / 32];
  double sum = 0.0;
  pdl_launch();
  for (int c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const int i = tensor_of(tab, c);
    const ClipTensor& t = tab.t[i];
    const bool last = c + 1 == (i + 1 < tab.count ? tab.t[i + 1].first : tab.chunks);
    sum += t.dt == MOE_F32 ? chunk_squares((const float*)t.g, t.numel, c - t.first, last)
                           : chunk_squares((const __nv_bfloat16*)t.g, t.numel, c - t.first, last);
  }
  sum = block_sum_f64(sum, red);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T* g, T* out, int64_t numel, int chunk, bool last, float f) {
  constexpr int V = Vec<T>::N;
  const int head = head_of(g, numel);
  const int64_t nvec = (numel - head) / V;
  const T* body = g + head;
  T* obody = out + head;
  const int64_t v0 = (int64_t)chunk * kChunkVec;
  const bool wide = ((uintptr_t)obody & 15u) == 0;      // out shares g's offset from a 16-byte boundary
  uint4 v[kChunkPer];
#pragma unroll
  for (int i = 0; i < kChunkPer; ++i) {
    const int64_t at = v0 + threadIdx.x + i * kClipThreads;
    if (at < nvec) v[i] = *reinterpret_cast<const uint4*>(body + at * V);
  }
#pragma unroll
  for (int i = 0; i < kChunkPer; ++i) {
    const int64_t at = v0 + threadIdx.x + i * kClipThreads;
    if (at >= nvec) continue;
    float x[V];
    Vec<T>::to_float(v[i], x);
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] *= f;
    if (wide) {
      st_v4(obody + at * V, Vec<T>::from_float(x));
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) obody[at * V + j] = from_f<T>(x[j]);
    }
  }
  if (chunk == 0 && (int)threadIdx.x < head) out[threadIdx.x] = from_f<T>(to_f<T>(g[threadIdx.x]) * f);
  if (last) {
    const int64_t at = head + nvec * V + threadIdx.x;
    if (at < numel) out[at] = from_f<T>(to_f<T>(g[at]) * f);
  }
}

// The same for a factor below a float's normal range, which would keep few of its bits there while
// g * f may well be normal: the products in double, an element at a time (nothing that a
// training step meets, and no registers for the vectors above).
template <typename T>
__device__ __forceinline__ void chunk_scale_tiny(const T* g, T* out, int64_t numel, int chunk, bool last, double f) {
  constexpr int64_t E = (int64_t)kChunkVec * Vec<T>::N;
  const int64_t end = last ? numel : (chunk + 1) * E;
#pragma unroll 1
  for (int64_t at = chunk * E + threadIdx.x; at < end; at += kClipThreads)
    out[at] = from_f<T>((float)((double)to_f<T>(g[at]) * f));
}

// The norm from the blocks' sums (in a fixed order, the same in every block),
// then the scaling.  The sums are still being written when this kernel starts: no restrict and no
// read-only path for them.  copy: the outputs are other buffers, written for f = 1 too.
template <int M>
__global__ void __launch_bounds__(kClipThreads)
grad_scale_kernel(const __grid_constant__ ClipTable<M> tab, const double* part, int n_part,
                  float max_norm, int copy, float* norm_out) {
  __shared__ double red[kClipThreads / 32];
  double sum = 0.0;
  pdl_wait();
  for (int i = threadIdx.x; i < n_part; i += 8 * kClipThreads) {     // eight loads in flight
    double v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j * kClipThreads < n_part ? part[i + j * kClipThreads] : 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += v[j];
  }
  const double norm = sqrt(block_sum_f64(sum, red));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  const double r = (double)max_norm / (norm + 1e-6);
  // a NaN norm stays visible in every gradient; without a limit nothing is scaled
  const float f = r >= 1.0 || isinf(max_norm) ? 1.0f : (float)r;
  if (f == 1.0f && !copy) return;
  for (int c = tab.chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
    const int i = tensor_of(tab, c);
    const ClipTensor& t = tab.t[i];
    const bool last = c + 1 == (i + 1 < tab.count ? tab.t[i + 1].first : tab.chunks);
    if (f < FLT_MIN) {
      if (t.dt == MOE_F32)
        chunk_scale_tiny((const float*)t.g, (float*)t.out, t.numel, c - t.first, last, r);
      else
        chunk_scale_tiny((const __nv_bfloat16*)t.g, (__nv_bfloat16*)t.out, t.numel, c - t.first, last, r);
    } else if (t.dt == MOE_F32)
      chunk_scale((const float*)t.g, (float*)t.out, t.numel, c - t.first, last, f);
    else
      chunk_scale((const __nv_bfloat16*)t.g, (__nv_bfloat16*)t.out, t.numel, c - t.first, last, f);
  }
}

inline size_t dt_bytes(int dt) { return dt == MOE_F32 ? 4 : 2; }

int64_t chunks_of(int64_t numel, int dt) {
  const int64_t c = cdiv(numel / (16 / (int64_t)dt_bytes(dt)), kChunkVec);
  return c > 0 ? c : 1;
}

// Two gradients that share memory, or an output that covers another
// gradient's input, would be scaled while a second block still reads them; so would
// what the call writes besides, the norm and the workspace.
bool overlapping(const void* const* grads, void* const* outs, const int64_t* numels, const int32_t* dts, int count,
                 const void* norm, const void* ws, size_t ws_bytes) {
  struct Range {
    uintptr_t a, b;
    int i;
  };
  std::vector<Range> w;
  w.reserve(count);
  for (int i = 0; i < count; ++i)
    if (numels[i] > 0) {
      const uintptr_t a = (uintptr_t)(outs ? outs[i] : grads[i]), bytes = (uintptr_t)numels[i] * dt_bytes(dts[i]);
      w.push_back({a, a + bytes, i});
      for (const uintptr_t p : {a, (uintptr_t)grads[i]})
        if (((uintptr_t)norm < p + bytes && p < (uintptr_t)norm + sizeof(float)) ||
            ((uintptr_t)ws < p + bytes && p < (uintptr_t)ws + ws_bytes))
          return true;
    }
  std::sort(w.begin(), w.end(), [](const Range& p, const Range& q) { return p.a < q.a; });
  for (size_t k = 1; k < w.size(); ++k)
    if (w[k].a < w[k - 1].b) return true;
  if (!outs) return false;
  for (int i = 0; i < count; ++i) {
    if (numels[i] == 0 || outs[i] == grads[i]) continue;
    const uintptr_t a = (uintptr_t)grads[i], b = a + (uintptr_t)numels[i] * dt_bytes(dts[i]);
    // the written ranges are disjoint and sorted: the last one starting before b
    auto it = std::lower_bound(w.begin(), w.end(), b, [](const Range& p, uintptr_t v) { return p.a < v; });
    if (it != w.begin() && (it - 1)->b > a) return true;
  }
  return false;
}

int launches_of(int count) { return count > 0 ? (int)cdiv(count, kClipMax) : 1; }

template <int M>
moe_status clip_run(const void* const* grads, void* const* outs, const int64_t* numels, const int32_t* dts,
                    int count, float max_norm, float* norm, double* part, cudaStream_t s) {
  ClipTable<M> tab;
  int n_part = 0;
  const bool copy = outs != nullptr;
  for (int pass = 0; pass < 2; ++pass) {
    int at = 0;
    bool first = true;
    while (first || at < count) {
      tab.count = 0;
      int64_t chunks = 0;
      while (at < count && tab.count < M) {
        if (numels[at] > 0) {
          const int64_t c = chunks_of(numels[at], dts[at]);
          if (chunks + c > 0x3fffffff) return MOE_ERR_UNSUPPORTED;
          tab.t[tab.count++] = {grads[at], copy ? outs[at] : const_cast<void*>(grads[at]), numels[at],
                                (int32_t)chunks, dts[at]};
          chunks += c;
        }
        ++at;
      }
      tab.chunks = (int32_t)chunks;
      const int blocks = chunks < kClipBlocks ? (int)chunks : kClipBlocks;
      if (pass == 0) {
        if (blocks > 0) {
          MOE_TRACED("grad_squares", s, (grad_squares_kernel<M><<<blocks, kClipThreads, 0, s>>>(tab, part + n_part)));
          MOE_LAUNCH_CHECK();
          n_part += blocks;
        }
      } else if (blocks > 0 || first) {
        cudaError_t err = cudaSuccess;
        MOE_TRACED("grad_scale", s,
                   (err = launch_after(grad_scale_kernel<M>, blocks > 0 ? blocks : 1, kClipThreads, 0, s, tab, part, n_part,
                                       max_norm, copy ? 1 : 0, first ? norm : nullptr)));
        if (err != cudaSuccess) {
          (void)cudaGetLastError();
          return MOE_ERR_CUDA;
        }
      }
      first = false;
    }
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_clip_grad_norm_workspace_size(int32_t count) {
  if (count < 0) return 0;
  return kStatusBytes + (size_t)launches_of(count) * kClipBlocks * sizeof(double);
}

moe_status moe_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* numels,
                              const int32_t* dtypes, int32_t count, float max_norm, float* norm, void* ws,
                              size_t ws_bytes, moe_stream_t stream) {
  if (count < 0 || !norm || !(max_norm >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (count > 0 && (!grads || !numels || !dtypes)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    if (dtypes[i] != MOE_F32 && dtypes[i] != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (numels[i] < 0) return MOE_ERR_INVALID_ARG;
    if (numels[i] == 0) continue;
    const uintptr_t mask = dt_bytes(dtypes[i]) - 1;
    if (!grads[i] || ((uintptr_t)grads[i] & mask)) return MOE_ERR_INVALID_ARG;
    if (outs && (!outs[i] || ((uintptr_t)outs[i] & mask))) return MOE_ERR_INVALID_ARG;
  }
  if (((uintptr_t)norm & 3u) || ((uintptr_t)ws & 15u)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < moe_clip_grad_norm_workspace_size(count)) return MOE_ERR_WORKSPACE;
  try {
    if (overlapping(grads, outs, numels, dtypes, count, norm, ws, moe_clip_grad_norm_workspace_size(count)))
      return MOE_ERR_INVALID_ARG;
  } catch (const std::bad_alloc&) {
    return MOE_ERR_UNSUPPORTED;   // no host memory for the check
  }
  double* part = (double*)((char*)ws + kStatusBytes);
  cudaStream_t s = (cudaStream_t)stream;
  // a short list takes a short parameter block: its launch copies 768 bytes, not 24 KB
  if (count <= 24) return clip_run<24>(grads, outs, numels, dtypes, count, max_norm, norm, part, s);
  if (count <= 128) return clip_run<128>(grads, outs, numels, dtypes, count, max_norm, norm, part, s);
  return clip_run<kClipMax>(grads, outs, numels, dtypes, count, max_norm, norm, part, s);
}

}  // extern "C"
