// Log probabilities of given tokens, with entropy and the most probable alternatives, and the
// gradient of the scores.
//
//   m = max x,  S = sum e^(x - m),  D = sum e^(x - m) (x - m)
//   ln p_j = x_j - m - ln S,  H = ln S - D / S
//   d_x_j = g ([j = token] - p_j) - h p_j (ln p_j + H)      g, h: gradients of ln p_token and H
//
// One pass over a row with the running maximum: a thread takes 32 scores at a time, and its sums
// move to the new maximum when these hold one. Differences x - m are formed before the exponential,
// so scores of any size (a mask of the type's lowest value among them) keep their meaning: -inf is no
// token, a row of nothing else has no distribution (S = 0).
#include "common.cuh"
#include "launch.cuh"
#include "ops.h"
#include "trace.h"

namespace moe {
namespace {

constexpr int LT = 512, LW = LT / 32;   // threads and warps of a block
constexpr float kLog2e = 1.44269504088896340736f, kLowest = -3.402823466e38f, kInf = __builtin_huge_valf();

// 2^x with an error of 2^-22 (numbers below 2^-126 count as 0)
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// the larger; NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// x - m, no lower than where e^(x - m) is 0 (so that 0 times it is 0 too)
__device__ __forceinline__ float below(float x, float m) { return max_nan(x - m, -200.f); }

// The sums of some scores: S = sum e^(x - m), D = sum e^(x - m) (x - m); none: m = kLowest, S = 0.
struct Sums {
  float m, S, D;
  __device__ __forceinline__ void to(float max) {   // the same sums about a maximum that is no lower
    const float d = below(m, max), e = exp2_fast(d * kLog2e);
    D = e * fmaf(d, S, D);
    S *= e;
    m = max;
  }
  __device__ __forceinline__ void join(Sums o) {
    const float max = fmaxf(m, o.m);
    to(max);
    o.to(max);
    S += o.S;
    D += o.D;
  }
};

// A score's place among the alternatives: higher score, then lower index. 0: no alternative.
__device__ __forceinline__ unsigned long long key_of(float x, uint32_t j) {
  const uint32_t b = __float_as_uint(x + 0.f);   // -0 is +0
  const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (unsigned long long)o << 32 | (0xffffffffu - j);
}
__device__ __forceinline__ uint32_t index_of(unsigned long long key) { return 0xffffffffu - (uint32_t)key; }

__device__ __forceinline__ unsigned long long max64(unsigned long long a, unsigned long long b) { return a > b ? a : b; }

template <typename T, bool VEC>
__device__ __forceinline__ void load_scores(float (&f)[8], const T* row, int j, int V, const T* end) {
  const int n = V - j;
  Vec8<T> v;
  if (VEC && n >= 8) {
    v.load_plain(row + j);
  } else if (!VEC) {
    load8_unaligned(v, row + j, end, n);
  } else {
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < n ? row[j + i] : T(0.f);
  }
  v.to_float(f);
  if (n < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= n) f[i] = -kInf;
  }
}

template <typename T, bool VEC, bool TOP>
__global__ void __launch_bounds__(LT) logprob_kernel(const LogprobArgs a) {
  __shared__ Sums s_sums[LW];
  __shared__ unsigned long long s_key[2][LW];
  constexpr int U = 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, V = a.V;
  pdl_start();
  pdl_wait();
  const int64_t m = blockIdx.x;
  const T* row = static_cast<const T*>(a.x) + m * a.ld;
  const T* end = static_cast<const T*>(a.x) + (a.M - 1) * a.ld + V;
  Sums s = {kLowest, 0.f, 0.f};
  unsigned long long best = 0;
  for (int j0 = threadIdx.x * 8; j0 < V; j0 += U * LT * 8) {
    float f[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * LT * 8;
      if (j < V) {
        load_scores<T, VEC>(f[u], row, j, V, end);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[u][i] = -kInf;
      }
    }
    float max = s.m;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) max = fmaxf(max, f[u][i]);
    s.to(max);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = below(f[u][i], max), e = exp2_fast(d * kLog2e);
        s.S += e;
        s.D = fmaf(e, d, s.D);
        if (TOP && f[u][i] > -kInf) best = max64(best, key_of(f[u][i], j0 + u * LT * 8 + i));
      }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums t;
    t.m = __shfl_xor_sync(0xffffffffu, s.m, o);
    t.S = __shfl_xor_sync(0xffffffffu, s.S, o);
    t.D = __shfl_xor_sync(0xffffffffu, s.D, o);
    s.join(t);
  }
  if (lane == 0) s_sums[warp] = s;
  __syncthreads();
  s = s_sums[lane % LW];
#pragma unroll
  for (int o = LW / 2; o > 0; o >>= 1) {
    Sums t;
    t.m = __shfl_xor_sync(0xffffffffu, s.m, o);
    t.S = __shfl_xor_sync(0xffffffffu, s.S, o);
    t.D = __shfl_xor_sync(0xffffffffu, s.D, o);
    s.join(t);
  }
  const float log_sum = s.S == 0.f ? -kInf : logf(s.S);   // a row without a distribution: -inf
  if (threadIdx.x == 0) {
    if (a.logprob != nullptr) {
      const int t = a.tokens[m];
      float lp = 0.f;
      if (t >= 0 && t < V) lp = s.S == 0.f ? -kInf : (to_f32(row[t]) - s.m) - log_sum;
      a.logprob[m] = lp;
    }
    if (a.stats != nullptr) reinterpret_cast<float2*>(a.stats)[m] = make_float2(s.m, log_sum);
    if (a.entropy != nullptr) a.entropy[m] = s.S == 0.f ? 0.f : log_sum - s.D / s.S;
  }
  if constexpr (TOP) {
    // the block's largest key, n times; its owner then looks for its next one
    for (int k = 0; k < a.n_top; ++k) {
      unsigned long long top = best;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = max64(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (lane == 0) s_key[k & 1][warp] = top;
      __syncthreads();
      top = s_key[k & 1][lane % LW];
#pragma unroll
      for (int o = LW / 2; o > 0; o >>= 1) top = max64(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int j = top == 0 ? -1 : (int)index_of(top);
      if (threadIdx.x == 0) {
        a.top_idx[m * a.n_top + k] = j;
        a.top_logprob[m * a.n_top + k] = j < 0 ? -kInf : (to_f32(row[j]) - s.m) - log_sum;
      }
      if (top != 0 && best == top) {
        best = 0;
        for (int j0 = threadIdx.x * 8; j0 < V; j0 += LT * 8)
          for (int i = 0; i < 8 && j0 + i < V; ++i) {
            const float x = to_f32(row[j0 + i]);
            const unsigned long long key = key_of(x, j0 + i);
            if (x > -kInf && key < top) best = max64(best, key);
          }
      }
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) logprob_bwd_kernel(const LogprobBwdArgs a) {
  const int V = a.V;
  pdl_start();
  pdl_wait();
  const int64_t m = blockIdx.x;
  const T* row = static_cast<const T*>(a.x) + m * a.ld;
  const T* end = static_cast<const T*>(a.x) + (a.M - 1) * a.ld + V;
  T* out = static_cast<T*>(a.dx) + m * a.ld_dx;
  const float2 st = reinterpret_cast<const float2*>(a.stats)[m];
  const bool some = !(st.y == -kInf);     // the row has a distribution
  const int token = a.d_logprob != nullptr && some ? a.tokens[m] : -1;
  const float g = token >= 0 && token < V ? a.d_logprob[m] : 0.f;
  const float h = a.d_entropy != nullptr && some ? a.d_entropy[m] : 0.f, H = h != 0.f ? a.entropy[m] : 0.f;
  const bool zero = g == 0.f && h == 0.f;
  for (int j = (blockIdx.y * 256 + threadIdx.x) * 8; j < V; j += gridDim.y * 2048) {
    float f[8];
    if (zero) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 0.f;
    } else {
      load_scores<T, VEC>(f, row, j, V, end);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float lp = below(f[i], st.x) - st.y, p = exp2_fast(lp * kLog2e);
        const float d = g * ((j + i == token ? 1.f : 0.f) - p);
        f[i] = h != 0.f ? d - h * (p * (lp + H)) : d;
      }
    }
    if (VEC && j + 8 <= V) {
      Vec8<T> v;
      v.from_float(f);
      v.store(out + j);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i < V) out[j + i] = from_f32<T>(f[i]);
    }
  }
}

template <typename T> cudaError_t logprob(const LogprobArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)a.M);
  const bool vec = a.M == 1 || a.ld % 8 == 0, top = a.n_top > 0;
  if (top) return vec ? launch_pdl(logprob_kernel<T, true, true>, grid, LT, 0, 1, st, a) : launch_pdl(logprob_kernel<T, false, true>, grid, LT, 0, 1, st, a);
  return vec ? launch_pdl(logprob_kernel<T, true, false>, grid, LT, 0, 1, st, a) : launch_pdl(logprob_kernel<T, false, false>, grid, LT, 0, 1, st, a);
}

template <typename T> cudaError_t logprob_bwd(const LogprobBwdArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)a.M, (unsigned)((a.V + 8191) / 8192));
  return a.M == 1 || (a.ld % 8 == 0 && a.ld_dx % 8 == 0) ? launch_pdl(logprob_bwd_kernel<T, true>, grid, 256, 0, 1, st, a)
                                           : launch_pdl(logprob_bwd_kernel<T, false>, grid, 256, 0, 1, st, a);
}

}  // namespace

cudaError_t launch_logprob(const LogprobArgs& a, int dtype, int num_sms, cudaStream_t st) {
  TraceScope ts(TP_LOGPROB, st);
  return dtype == MOE_F32 ? logprob<float>(a, st) : logprob<__nv_bfloat16>(a, st);
}

cudaError_t launch_logprob_bwd(const LogprobBwdArgs& a, int dtype, cudaStream_t st) {
  TraceScope ts(TP_LOGPROB_BWD, st);
  return dtype == MOE_F32 ? logprob_bwd<float>(a, st) : logprob_bwd<__nv_bfloat16>(a, st);
}

}  // namespace moe
