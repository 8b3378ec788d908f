// The global norm of many gradients, and their clipping to a largest norm.
//
//   norm = sqrt(sum over all tensors of sum x^2),  scale = min(1, max_norm / (norm + 1e-6)),  out = x scale
//
// Two passes over the gradients (the scale is known after the first), both bound by HBM. The tensors
// are cut into chunks of 32 KB, which the blocks take in turn, whatever the tensors' sizes; the
// second pass takes them from the last one back, and finds in L2 a part of what the first one read last (42 MB of 200:
// 100M bf16, of which it reads 158 from DRAM).
// A thread adds the squares of its 128 bytes in fp32 and those sums in pairs of fp32 numbers (the second
// one what rounding the first took away: fp64 runs at a sixtieth of fp32's rate); the blocks' sums are
// written out and added in order, so a result does not depend on timing. Squares that leave fp32's
// range (a thread's sum beyond 2^90, or below 2^-60) are taken in fp64 again.
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

// The tensor that a chunk belongs to; `first`: the table's, in shared memory (every 16th one first, then
// those between). Chunks begin at a 16-byte boundary of the tensor's memory (the elements before the first one
// belong to its chunk 0).
static_assert(kClipMany <= 32 * 16, "");
__device__ __forceinline__ int tensor_of(const uint32_t* first, int count, uint32_t chunk) {
  const int lane = threadIdx.x & 31, i = lane * 16;
  const int base = (__popc(__ballot_sync(0xffffffffu, i < count && first[i] <= chunk)) - 1) * 16, k = base + 1 + lane;
  return base + __popc(__ballot_sync(0xffffffffu, lane < 15 && k < count && first[k] <= chunk));
}
template <int CAP> __device__ __forceinline__ void share_first(const ClipTable<CAP>& t, uint32_t* first) {
  for (int i = threadIdx.x; i <= t.count; i += CT) first[i] = t.first[i];
  __syncthreads();
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
      if (j + W <= n) {
        v[u] = *reinterpret_cast<const uint4*>(p + j);
      } else {
        T* e = reinterpret_cast<T*>(&v[u]);
#pragma unroll
        for (int i = 0; i < W; ++i) e[i] = j + i < n ? p[j + i] : T(0.f);
      }
    }
  }
}

// A chunk of a tensor, looked up while the one before is on its way.
struct Chunk {
  const void* g;
  int64_t n, local;
  int tensor;
  bool f32;
};
template <int CAP> __device__ __forceinline__ Chunk chunk_at(const ClipTable<CAP>& t, const uint32_t* first, uint32_t c) {
  const int i = tensor_of(first, t.count, c);
  return {t.g[i], t.n[i], (int64_t)(c - first[i]), i, t.f32[i] != 0};
}

// A sum of numbers in [2^-60, 2^90] as hi + lo, with an error of a few 2^-48, and of others in fp64.
struct Total {
  float hi, lo;
  double far;
  __device__ __forceinline__ void add(float h, float l) {   // (rounding errors of a sum: Knuth's two-sum)
    const float s = hi + h, b = s - hi;
    lo += l + ((hi - (s - b)) + (h - b));
    hi = s;
  }
};

__device__ __forceinline__ bool some(double far) { return __double_as_longlong(far) != 0; }   // (no fp64 comparison)

// The squares of a chunk's elements (load_chunk's vectors, and what stands before the first one).
template <typename T> __device__ __forceinline__ void add_squares(Total& total, const uint4 (&v)[CU], float head) {
  constexpr int W = kVec<T>;
  float s[2] = {head * head, 0.f};
#pragma unroll
  for (int u = 0; u < CU; ++u) {
    float f[W];
    vec_floats(v[u], f, T());
#pragma unroll
    for (int i = 0; i < W; ++i) s[i & 1] = fmaf(f[i], f[i], s[i & 1]);
  }
  const float t = s[0] + s[1];
  if (t >= 0x1p-60f && t <= 0x1p90f) {
    total.add(t, 0.f);
    return;
  }
  if (t == 0.f) {   // mostly because all of them are 0 (an expert without tokens): no fp64 for that
    uint32_t bits = head != 0.f;
#pragma unroll
    for (int u = 0; u < CU; ++u) bits |= v[u].x | v[u].y | v[u].z | v[u].w;
    if ((bits & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu)) == 0u) return;
  }
  double d = total.far;
  if (head != 0.f) d = fma((double)head, (double)head, d);
#pragma unroll
  for (int u = 0; u < CU; ++u) {
    float f[W];
    vec_floats(v[u], f, T());
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (f[i] != 0.f) d = fma((double)f[i], (double)f[i], d);
  }
  total.far = d;
}
// Where this thread's vectors of a chunk begin.
template <typename T> __device__ __forceinline__ int64_t chunk_start(const T* p, int64_t n, int64_t chunk) {
  return head_of(p, n) + chunk * (CB / (int)sizeof(T)) + threadIdx.x * kVec<T>;
}

__device__ __forceinline__ void over_lanes(Total& t) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float h = __shfl_xor_sync(0xffffffffu, t.hi, o), l = __shfl_xor_sync(0xffffffffu, t.lo, o);
    t.add(h, l);
  }
  if (__any_sync(0xffffffffu, some(t.far))) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t.far += __shfl_xor_sync(0xffffffffu, t.far, o);
  }
}

// The block's sum, in every thread.
__device__ __forceinline__ void over_block(Total& t) {
  __shared__ Total s[CT / 32];
  over_lanes(t);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = t;
  __syncthreads();
  t = s[0];
#pragma unroll
  for (int w = 1; w < CT / 32; ++w) {
    t.add(s[w].hi, s[w].lo);
    if (some(s[w].far)) t.far += s[w].far;
  }
}

// norm and scale from the blocks' sums, the same in every thread.
__device__ __forceinline__ void norm_scale(const ClipPart* part, int n_part, float max_norm, float& norm, float& scale) {
  Total t = {0.f, 0.f, 0.0};
  constexpr int U = 2;   // parts of a thread that are under way
  for (int i0 = threadIdx.x; i0 < n_part; i0 += CT * U) {
    ClipPart p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      p[u] = {0.f, 0.f, 0.0};
      if (i0 + CT * u < n_part) *reinterpret_cast<uint4*>(&p[u]) = __ldcg(reinterpret_cast<const uint4*>(part + i0 + CT * u));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      t.add(p[u].hi, p[u].lo);
      if (some(p[u].far)) t.far += p[u].far;
    }
  }
  over_block(t);
  if (some(t.far)) {
    const double d = sqrt((double)t.hi + (double)t.lo + t.far), q = (double)max_norm / (d + 1e-6);
    norm = (float)d;
    scale = q >= 1.0 ? 1.f : (float)q;   // NaN stays
  } else {
    // sqrt(hi) and a Newton step towards the root of hi + lo
    float r = sqrtf(t.hi);
    if (r > 0.f) r += (fmaf(-r, r, t.hi) + t.lo) / (2.f * r);
    const float q = max_norm / (r + 1e-6f);
    norm = r;
    scale = q >= 1.f ? 1.f : q;
  }
  if (max_norm == __builtin_huge_valf()) scale = 1.f;
}

// Squares of all chunks. 571M bf16: 160 us, 7.1 TB/s; 300 tensors of 111M elements 36 us (51 while chunks that end a
// tensor went through fp64 for their zeros); 3.1M fp32 6.7 us, launch, load and the blocks' join. 80 registers and 26 bytes spilled, for three blocks on an SM.
// A launch's sums go to part[first ..]. counter: its blocks that are done, where this is the call's last
// launch (the last block then writes norm and scale), else NULL.
template <int CAP>
__global__ void __launch_bounds__(CT, kClipBlocks) clip_squares_kernel(const __grid_constant__ ClipTable<CAP> t, ClipPart* part, int first,
                                                                       uint32_t* counter, float max_norm, float* norm, float* scale) {
  __shared__ uint32_t s_first[CAP + 1];
  __shared__ bool s_last;
  pdl_start();
  share_first(t, s_first);
  pdl_wait();
  const uint32_t chunks = s_first[t.count];
  Total total = {0.f, 0.f, 0.0};
  uint32_t c = blockIdx.x;
  Chunk k = {};
  if (c < chunks) k = chunk_at(t, s_first, c);
  while (c < chunks) {
    const bool f32 = k.f32;
    uint4 v[CU];
    float head = 0.f;   // what stands before the first 16-byte boundary
    if (f32) {
      const float* p = static_cast<const float*>(k.g);
      load_chunk(v, p, chunk_start(p, k.n, k.local), k.n);
      if (k.local == 0 && threadIdx.x < head_of(p, k.n)) head = p[threadIdx.x];
    } else {
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(k.g);
      load_chunk(v, p, chunk_start(p, k.n, k.local), k.n);
      if (k.local == 0 && threadIdx.x < head_of(p, k.n)) head = to_f32(p[threadIdx.x]);
    }
    c += gridDim.x;
    if (c < chunks) k = chunk_at(t, s_first, c);
    if (f32) add_squares<float>(total, v, head);
    else add_squares<__nv_bfloat16>(total, v, head);
  }
  over_block(total);
  if (threadIdx.x == 0) part[first + blockIdx.x] = {total.hi, total.lo, total.far};
  if (counter == nullptr) return;
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(counter, 1u) + 1 == gridDim.x;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  float n, s;
  norm_scale(part, first + (int)gridDim.x, max_norm, n, s);
  if (threadIdx.x == 0) {
    if (norm != nullptr) *norm = n;
    if (scale != nullptr) *scale = s;
    *counter = 0;
  }
}

// A chunk's vectors, loaded by load_chunk, on their way out.
template <typename T>
__device__ __forceinline__ void scale_chunk(const uint4 (&v)[CU], const T* p, T* out, int64_t n, int64_t chunk, float scale) {
  constexpr int W = kVec<T>;
  const int h = head_of(p, n);
  const int64_t at = h + chunk * (CB / sizeof(T)) + threadIdx.x * W;
  const bool vec = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  if (chunk == 0 && threadIdx.x < h) out[threadIdx.x] = from_f32<T>(to_f32(p[threadIdx.x]) * scale);
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
}

// The second pass. 571M bf16: 360 us for a read and a write of each, 6.4 TB/s. A result that begins at another place within 16
// bytes than its gradient goes out by single elements: 100M bf16 clipped into another tensor 92 us, 308 one element off.
// part: the blocks' sums of every launch of the first pass; block 0 writes norm and scale. A block's first
// chunk is under way while it works out the scale.
template <int CAP>
__global__ void __launch_bounds__(CT, kClipBlocks) clip_scale_kernel(const __grid_constant__ ClipTable<CAP> t, const ClipPart* part, int n_part,
                                                                     float max_norm, float* norm, float* scale_out) {
  __shared__ uint32_t s_first[CAP + 1];
  pdl_start();
  share_first(t, s_first);
  pdl_wait();
  const uint32_t chunks = s_first[t.count];
  uint4 v[CU];
  float scale = 0.f;
  bool known = false;
  uint32_t left = blockIdx.x;   // from the last chunk back
  Chunk k = {};
  if (left < chunks) k = chunk_at(t, s_first, chunks - 1 - left);
  while (left < chunks) {
    const Chunk now = k;
    const float* pf = static_cast<const float*>(now.g);
    const __nv_bfloat16* pb = static_cast<const __nv_bfloat16*>(now.g);
    void* out = t.out[now.tensor];
    left += gridDim.x;
    if (known && (out == nullptr || (scale == 1.f && out == now.g))) {
      if (left < chunks) k = chunk_at(t, s_first, chunks - 1 - left);
      continue;
    }
    if (now.f32) load_chunk(v, pf, chunk_start(pf, now.n, now.local), now.n);
    else load_chunk(v, pb, chunk_start(pb, now.n, now.local), now.n);
    if (left < chunks) k = chunk_at(t, s_first, chunks - 1 - left);
    if (!known) {
      float value;
      norm_scale(part, n_part, max_norm, value, scale);
      if (threadIdx.x == 0 && blockIdx.x == 0) {
        if (norm != nullptr) *norm = value;
        if (scale_out != nullptr) *scale_out = scale;
      }
      known = true;
      if (out == nullptr || (scale == 1.f && out == now.g)) continue;
    }
    if (now.f32) scale_chunk(v, pf, static_cast<float*>(out), now.n, now.local, scale);
    else scale_chunk(v, pb, static_cast<__nv_bfloat16*>(out), now.n, now.local, scale);
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
  for (int64_t i = 0; i < a.count; ++i) write |= a.grads[i].out != nullptr && a.grads[i].n > 0;
  int64_t at = 0;
  do {   // (once at least: no tensors have a norm too)
    at = fill(t, a.grads, at, a.count);
    const uint32_t chunks = t.first[t.count], grid = chunks < 1 ? 1 : chunks < most ? chunks : most;
    const cudaError_t e = launch_pdl(clip_squares_kernel<CAP>, dim3(grid), CT, 0, 1, st, t, a.part, n_part,
                                     !write && at == a.count ? a.counter : nullptr, a.max_norm, a.norm, a.scale);
    if (e != cudaSuccess) return e;
    n_part += (int)grid;
  } while (at < a.count);
  if (!write) return cudaSuccess;
  for (at = 0; at < a.count;) {
    at = fill(t, a.grads, at, a.count);
    const uint32_t chunks = t.first[t.count], grid = chunks < most ? chunks : most;
    if (chunks == 0) continue;
    const cudaError_t e = launch_pdl(clip_scale_kernel<CAP>, dim3(grid), CT, 0, 1, st, t, (const ClipPart*)a.part, n_part, a.max_norm,
                                     a.norm, a.scale);
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
