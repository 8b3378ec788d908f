// The global norm of many gradients, and their clipping to a largest norm.
//
//   norm = sqrt(sum over all tensors of sum x^2),  scale = min(1, max_norm / (norm + 1e-6)),  out = x scale
//
// Two passes over the gradients (the scale is known after the first), both bound by HBM. The tensors
// are cut into chunks of 16384 elements, which the blocks take in turn, whatever the tensors' sizes.
// A thread adds the squares of 64 elements in fp32 and those sums in fp64; the blocks' sums are
// written out and added in order, so a result does not depend on timing. Squares that leave fp32's
// range (elements beyond 2^63, or a chunk below 2^-30) are taken in fp64 again.
#include <math.h>

#include "common.cuh"
#include "launch.cuh"
#include "ops.h"
#include "trace.h"

namespace moe {
namespace {

constexpr int CT = 256, CE = CT * 64;   // threads of a block, elements of a chunk

template <int CAP> struct ClipTable {
  const void* g[CAP];
  void* out[CAP];
  int64_t n[CAP];
  uint32_t first[CAP + 1];   // chunk of the launch that a tensor begins with
  uint8_t f32[CAP];
  int count;
};

// A chunk's tensor and its first element there. Chunks begin at a 16-byte boundary of the tensor's memory
// (the elements before the first one belong to chunk 0).
template <int CAP> __device__ __forceinline__ int tensor_of(const ClipTable<CAP>& t, uint32_t chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
template <typename T> __device__ __forceinline__ int head_of(const T* p, int64_t n) {
  const int h = (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(T);
  return h < n ? h : (int)n;
}

__device__ __forceinline__ double square(double x) { return x * x; }

// The squares of a chunk's elements, this thread's share.
template <typename T> __device__ __forceinline__ double chunk_squares(const T* p, int64_t n, int64_t chunk) {
  constexpr int U = 8;
  const int h = head_of(p, n);
  const int64_t at = h + chunk * CE;
  Vec8<T> v[U];
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t j = at + (u * CT + threadIdx.x) * 8;
    if (j + 8 <= n) {
      v[u].load_plain(p + j);
    } else {
      T* e = reinterpret_cast<T*>(&v[u]);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = j + i < n ? p[j + i] : T(0.f);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float f[8];
    v[u].to_float(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(f[i], f[i], s);
  }
  double d = s;
  if (!(s >= 0x1p-60f && s <= 0x1p126f)) {   // (s = 0 mostly because all of them are)
    d = 0.0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[8];
      v[u].to_float(f);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (f[i] != 0.f) d += square((double)f[i]);
    }
  }
  if (chunk == 0 && threadIdx.x < h) d += square((double)to_f32(p[threadIdx.x]));
  return d;
}

// The same sum over the block in every thread.
__device__ __forceinline__ double block_sum(double d, double* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = d;
  __syncthreads();
  d = 0.0;
#pragma unroll
  for (int w = 0; w < CT / 32; ++w) d += s[w];
  return d;
}

template <int CAP> __global__ void __launch_bounds__(CT) clip_squares_kernel(const __grid_constant__ ClipTable<CAP> t, double* part) {
  __shared__ double s[CT / 32];
  pdl_start();
  pdl_wait();
  const uint32_t chunks = t.first[t.count];
  double d = 0.0;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t local = c - t.first[i];
    d += t.f32[i] ? chunk_squares(static_cast<const float*>(t.g[i]), t.n[i], local)
                  : chunk_squares(static_cast<const __nv_bfloat16*>(t.g[i]), t.n[i], local);
  }
  d = block_sum(d, s);
  if (threadIdx.x == 0) part[blockIdx.x] = d;
}

template <typename T> __device__ __forceinline__ void scale_chunk(const T* p, T* out, int64_t n, int64_t chunk, float scale) {
  constexpr int U = 8;
  const int h = head_of(p, n);
  const int64_t at = h + chunk * CE;
  const bool vec = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  Vec8<T> v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t j = at + (u * CT + threadIdx.x) * 8;
    if (j + 8 <= n) {
      v[u].load_plain(p + j);
    } else {
      T* e = reinterpret_cast<T*>(&v[u]);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = j + i < n ? p[j + i] : T(0.f);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t j = at + (u * CT + threadIdx.x) * 8;
    float f[8];
    v[u].to_float(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= scale;
    if (vec && j + 8 <= n) {
      v[u].from_float(f);
      v[u].store(out + j);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i < n) out[j + i] = from_f32<T>(f[i]);
    }
  }
  if (chunk == 0 && threadIdx.x < h) out[threadIdx.x] = from_f32<T>(to_f32(p[threadIdx.x]) * scale);
}

// part: the blocks' sums of every launch of the first pass; block 0 writes norm and scale.
template <int CAP>
__global__ void __launch_bounds__(CT) clip_scale_kernel(const __grid_constant__ ClipTable<CAP> t, const double* part, int n_part, float max_norm,
                                                       float* norm, float* scale_out) {
  __shared__ double s[CT / 32];
  pdl_start();
  pdl_wait();
  double d = 0.0;
  for (int i = threadIdx.x; i < n_part; i += CT) d += part[i];
  d = sqrt(block_sum(d, s));
  const double q = (double)max_norm / (d + 1e-6);
  const float scale = max_norm == __builtin_huge_valf() || q >= 1.0 ? 1.f : (float)q;   // NaN stays
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (norm != nullptr) *norm = (float)d;
    if (scale_out != nullptr) *scale_out = scale;
  }
  const uint32_t chunks = t.first[t.count];
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    if (t.out[i] == nullptr || (scale == 1.f && t.out[i] == t.g[i])) continue;
    const int64_t local = c - t.first[i];
    if (t.f32[i]) scale_chunk(static_cast<const float*>(t.g[i]), static_cast<float*>(t.out[i]), t.n[i], local, scale);
    else scale_chunk(static_cast<const __nv_bfloat16*>(t.g[i]), static_cast<__nv_bfloat16*>(t.out[i]), t.n[i], local, scale);
  }
}

// Tensors of one launch, from grads[at] on; returns where the next one begins.
template <int CAP> int64_t fill(ClipTable<CAP>& t, const moe_grad* grads, int64_t at, int64_t count) {
  t.count = 0;
  t.first[0] = 0;
  for (; at < count && t.count < CAP; ++at) {
    const moe_grad& g = grads[at];
    if (g.n == 0) continue;
    const int k = t.count++;
    t.g[k] = g.g;
    t.out[k] = g.out;
    t.n[k] = g.n;
    t.f32[k] = g.dtype == MOE_F32;
    t.first[k + 1] = t.first[k] + (uint32_t)((g.n + CE - 1) / CE);   // (below 2^31: kClipMaxTotal)
  }
  return at;
}

template <int CAP>
cudaError_t clip(const ClipArgs& a, int num_sms, cudaStream_t st) {
  ClipTable<CAP> t;
  int n_part = 0;
  const uint32_t most = (uint32_t)(num_sms * 4 < kClipParts ? num_sms * 4 : kClipParts);
  bool write = false;
  for (int64_t at = 0; at < a.count;) {
    at = fill(t, a.grads, at, a.count);
    if (t.count == 0) continue;
    const uint32_t chunks = t.first[t.count], grid = chunks < most ? chunks : most;
    const cudaError_t e = launch_pdl(clip_squares_kernel<CAP>, dim3(grid), CT, 0, 1, st, t, a.part + n_part);
    if (e != cudaSuccess) return e;
    n_part += grid;
  }
  for (int64_t i = 0; i < a.count; ++i) write |= a.grads[i].out != nullptr && a.grads[i].n > 0;
  if (!write) {
    t.count = 0;
    t.first[0] = 0;
    return launch_pdl(clip_scale_kernel<CAP>, dim3(1), CT, 0, 1, st, t, (const double*)a.part, n_part, a.max_norm, a.norm, a.scale);
  }
  for (int64_t at = 0; at < a.count;) {
    at = fill(t, a.grads, at, a.count);
    if (t.count == 0) continue;
    const uint32_t chunks = t.first[t.count], grid = chunks < most ? chunks : most;
    const cudaError_t e = launch_pdl(clip_scale_kernel<CAP>, dim3(grid), CT, 0, 1, st, t, (const double*)a.part, n_part, a.max_norm, a.norm, a.scale);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_clip(const ClipArgs& a, int num_sms, cudaStream_t st) {
  TraceScope ts(TP_CLIP, st);
  return a.count <= kClipFew ? clip<kClipFew>(a, num_sms, st) : clip<kClipMany>(a, num_sms, st);
}

}  // namespace moe
