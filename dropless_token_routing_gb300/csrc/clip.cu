// The global norm of many gradients, and their clipping to a largest norm.
//
//   norm = sqrt(sum over all tensors of sum x^2),  scale = min(1, max_norm / (norm + 1e-6)),  out = x scale
//
// Two passes over the gradients (the scale is known after the first), both bound by HBM. The tensors
// are cut into chunks of 32 KB, which the blocks take in turn, whatever the tensors' sizes; the
// second pass takes them from the last one back, so that it finds in L2 what the first one read last.
// A thread adds the squares of its 128 bytes in fp32 and those sums in fp64; the blocks' sums are
// written out and added in order, so a result does not depend on timing. Squares that leave fp32's
// range (elements beyond 2^63, or all of a thread's below 2^-33) are taken in fp64 again.
#include <math.h>

#include "common.cuh"
#include "launch.cuh"
#include "ops.h"
#include "trace.h"

namespace moe {
namespace {

constexpr int CT = 256, CU = 8, CB = CT * CU * 16;   // threads of a block, 16-byte vectors of a thread, bytes of a chunk
constexpr int kClipBlocks = 3;   // of an SM
template <typename T> constexpr int kVec = 16 / sizeof(T);   // elements of a vector

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

__device__ __forceinline__ void vec_floats(const uint4& v, float (&f)[4], float) {
  f[0] = __uint_as_float(v.x);
  f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z);
  f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void vec_floats(const uint4& v, float (&f)[8], __nv_bfloat16) {
  Vec8<__nv_bfloat16> b;
  b.v = v;
  b.to_float(f);
}
__device__ __forceinline__ uint4 floats_vec(const float (&f)[4], float) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 floats_vec(const float (&f)[8], __nv_bfloat16) {
  Vec8<__nv_bfloat16> b;
  b.from_float(f);
  return b.v;
}

// This thread's vectors of a chunk: vector u begins at element `at` + u * CT * kVec (zeros past n).
template <typename T> __device__ __forceinline__ void load_chunk(uint4 (&v)[CU], const T* p, int64_t at, int64_t n) {
  constexpr int W = kVec<T>;
  if (at + (CU - 1) * CT * W + W <= n) {
#pragma unroll
    for (int u = 0; u < CU; ++u) v[u] = *reinterpret_cast<const uint4*>(p + at + u * CT * W);
  } else {
#pragma unroll
    for (int u = 0; u < CU; ++u) {
      const int64_t j = at + u * CT * W;
      T* e = reinterpret_cast<T*>(&v[u]);
#pragma unroll
      for (int i = 0; i < W; ++i) e[i] = j + i < n ? p[j + i] : T(0.f);
    }
  }
}

// The squares of a chunk's elements, this thread's share.
template <typename T> __device__ __forceinline__ double chunk_squares(const T* p, int64_t n, int64_t chunk) {
  constexpr int W = kVec<T>;
  const int h = head_of(p, n);
  uint4 v[CU];
  load_chunk(v, p, h + chunk * (CB / sizeof(T)) + threadIdx.x * W, n);
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int u = 0; u < CU; ++u) {
    float f[W];
    vec_floats(v[u], f, T());
#pragma unroll
    for (int i = 0; i < W; ++i) s[i & 1] = fmaf(f[i], f[i], s[i & 1]);
  }
  const float t = s[0] + s[1];
  double d = t;
  if (!(t >= 0x1p-60f && t <= 0x1p126f)) {   // (t = 0 mostly because all of them are)
    d = 0.0;
#pragma unroll
    for (int u = 0; u < CU; ++u) {
      float f[W];
      vec_floats(v[u], f, T());
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (f[i] != 0.f) d = fma((double)f[i], (double)f[i], d);
    }
  }
  if (chunk == 0 && threadIdx.x < h) {
    const double x = to_f32(p[threadIdx.x]);
    d = fma(x, x, d);
  }
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

template <int CAP> __global__ void __launch_bounds__(CT, kClipBlocks) clip_squares_kernel(const __grid_constant__ ClipTable<CAP> t, double* part) {
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
  constexpr int W = kVec<T>;
  const int h = head_of(p, n);
  const int64_t at = h + chunk * (CB / sizeof(T)) + threadIdx.x * W;
  const bool vec = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  uint4 v[CU];
  load_chunk(v, p, at, n);
#pragma unroll
  for (int u = 0; u < CU; ++u) {
    const int64_t j = at + u * CT * W;
    float f[W];
    vec_floats(v[u], f, T());
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] *= scale;
    if (vec && j + W <= n) {
      *reinterpret_cast<uint4*>(out + j) = floats_vec(f, T());
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (j + i < n) out[j + i] = from_f32<T>(f[i]);
    }
  }
  if (chunk == 0 && threadIdx.x < h) out[threadIdx.x] = from_f32<T>(to_f32(p[threadIdx.x]) * scale);
}

// part: the blocks' sums of every launch of the first pass; block 0 writes norm and scale.
template <int CAP>
__global__ void __launch_bounds__(CT, kClipBlocks) clip_scale_kernel(const __grid_constant__ ClipTable<CAP> t, const double* part, int n_part, float max_norm,
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
  for (uint32_t k = blockIdx.x; k < chunks; k += gridDim.x) {
    const uint32_t c = chunks - 1 - k;
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
    const int64_t e = CB / (int64_t)elt_bytes(g.dtype);
    t.first[k + 1] = t.first[k] + (uint32_t)((g.n + e - 1) / e);   // (below 2^32: kClipMaxTotal)
  }
  return at;
}

template <int CAP>
cudaError_t clip(const ClipArgs& a, int num_sms, cudaStream_t st) {
  ClipTable<CAP> t;
  int n_part = 0;
  const uint32_t most = (uint32_t)(num_sms * kClipBlocks < kClipParts ? num_sms * kClipBlocks : kClipParts);   // all at once
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
