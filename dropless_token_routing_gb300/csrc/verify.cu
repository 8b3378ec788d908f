// Verification of drafted tokens: which of them stay, and the token drawn after the last one
// that stays.
//
// Only one row of the target's probabilities (and one of the draft's) is read per sequence: the
// row at the first refusal, or the one after the last kept token. Its weights are whole
// multiples of 2^-40 and are summed as 64-bit integers, so the sums, and with them the drawn
// token, do not depend on how the row is split over threads and CTAs.
//
// A sequence is a cluster: every CTA finds the first refusal itself (that is cheaper than telling the
// others), the CTAs share the row and exchange their sums. Bound by latency for few sequences (tokens,
// their probabilities, the row, the sums, the drawn chunk, each a wait for the one before), by HBM
// for many: B = 1, V = 32000: 5.2 us; B = 16, V = 50001: 8.1 us; B = 128, V = 131072 in fp32: 134 MB in
// 34 us, 3.9 TB/s.
#include "cluster.cuh"
#include "common.cuh"
#include "launch.cuh"
#include "ops.h"
#include "trace.h"

namespace moe {
namespace {

constexpr int VT = 512, VW = VT / 32;   // threads and warps per CTA

// An fp32 weight as a whole number of 2^-40, added to two sums of 2^-20 and 2^-40 (32 bits each:
// below 2^12 weights). fmaxf takes NaN to 0. Truncation by adding 2^23 towards zero: every step is
// exact or truncates, at the full fp32 rate (with 64-bit conversions the largest case takes 62 us, not
// 34).
__device__ __forceinline__ void add_mass(float r, uint32_t& hi, uint32_t& lo) {
  constexpr float k20 = 1048576.f, k23 = 8388608.f;
  const float x = fminf(fmaxf(r, 0.f), 1.f) * k20;
  const float h = __fadd_rz(x, k23);
  const float l = __fadd_rz((x - (h - k23)) * k20, k23);
  hi += __float_as_uint(h) & 0x7fffffu;
  lo += __float_as_uint(l) & 0x7fffffu;
}
__device__ __forceinline__ long long joined(uint32_t hi, uint32_t lo) { return ((long long)hi << 20) + lo; }

// A row's weights, a chunk of 32 lanes x W elements at a time: W neighbouring elements per lane
// (16 bytes) where both rows are aligned, else one.
template <typename T, bool VEC> struct Row {
  static constexpr int W = VEC ? 16 / sizeof(T) : 1;
  static constexpr int CHUNK = 32 * W;
  const T *p, *q;   // q NULL: p alone
  int V;
  struct Raw {
    T p[W], q[W];
  };
  __device__ __forceinline__ static void load(T (&d)[W], const T* s) {
    if constexpr (VEC) *reinterpret_cast<uint4*>(d) = *reinterpret_cast<const uint4*>(s);
    else d[0] = s[0];
  }
  // elements j .. j + W - 1 (all of them past V count as 0; with VEC, V may end inside)
  template <bool Q> __device__ __forceinline__ void get(Raw& r, int j) const {
    if (j + W <= V) {
      load(r.p, p + j);
      if (Q) load(r.q, q + j);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        r.p[i] = j + i < V ? p[j + i] : from_f32<T>(0.f);
        if (Q) r.q[i] = j + i < V ? q[j + i] : from_f32<T>(0.f);
      }
    }
  }
  template <bool Q> __device__ __forceinline__ static float weight(const Raw& r, int i) {
    return Q ? to_f32(r.p[i]) - to_f32(r.q[i]) : to_f32(r.p[i]);
  }
  template <bool Q> __device__ __forceinline__ static void add(const Raw& r, uint32_t& hi, uint32_t& lo) {
#pragma unroll
    for (int i = 0; i < W; ++i) add_mass(weight<Q>(r, i), hi, lo);
  }
  // this lane's sum of elements [j0, j1), U chunks in flight
  template <bool Q> __device__ __forceinline__ long long total(int j0, int j1, int lane) const {
    constexpr int U = !VEC ? 8 : sizeof(T) == 4 ? 4 : 2;
    long long s = 0;
    for (int j = j0; j < j1; j += U * CHUNK) {
      alignas(16) Raw r[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int at = j + i * CHUNK + lane * W;
        get<Q>(r[i], at < j1 ? at : V);
      }
      uint32_t hi = 0, lo = 0;
#pragma unroll
      for (int i = 0; i < U; ++i) add<Q>(r[i], hi, lo);
      s += joined(hi, lo);
    }
    return s;
  }
  // The element of [j0, j1) where the sums, from `cum` on, pass `level` (it is there).
  template <bool Q> __device__ __forceinline__ int find(int j0, int j1, long long cum, long long level, int lane) const {
    for (int j = j0; j < j1; j += 32 * CHUNK) {
      // lane i: the sum of chunk i of 32
      long long mine = 0;
      const int chunks = min(32, (j1 - j + CHUNK - 1) / CHUNK);
#pragma unroll 4
      for (int i = 0; i < chunks; ++i) {
        const int at = j + i * CHUNK + lane * W;
        alignas(16) Raw r;
        get<Q>(r, at < j1 ? at : V);
        uint32_t hi = 0, lo = 0;
        add<Q>(r, hi, lo);
        hi = __reduce_add_sync(0xffffffffu, hi);
        lo = __reduce_add_sync(0xffffffffu, lo);
        if (lane == i) mine = joined(hi, lo);
      }
      long long inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, cum + inc > level);
      if (past == 0u) {
        cum += __shfl_sync(0xffffffffu, inc, 31);
        continue;
      }
      const int c = __ffs((int)past) - 1;
      cum += __shfl_sync(0xffffffffu, inc - mine, c);
      const int at = j + c * CHUNK + lane * W;
      alignas(16) Raw r;
      get<Q>(r, at < j1 ? at : V);
      uint32_t hi = 0, lo = 0;
      add<Q>(r, hi, lo);
      const long long s = joined(hi, lo);
      inc = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
      }
      const int l = __ffs((int)__ballot_sync(0xffffffffu, cum + inc > level)) - 1;
      int e = 0;
      if constexpr (W > 1) {   // within lane l
        long long before = cum + inc - s;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          uint32_t h = 0, g = 0;
          add_mass(weight<Q>(r, i), h, g);
          before += joined(h, g);
          if (before <= level) e = i + 1;
        }
      }
      return __shfl_sync(0xffffffffu, at + e, l);
    }
    return -1;
  }
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(VT, 2) verify_kernel(const VerifyArgs v) {
  __shared__ int s_a, s_len;
  __shared__ long long s_sum[2][VW];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ctarank(), nrank = nctarank();
  pdl_start();
  pdl_wait();
  const int64_t b = blockIdx.x / nrank;
  const int n = v.n, V = v.V;
  const T* q0 = static_cast<const T*>(v.q) + b * n * v.ld_q;
  const T* p0 = static_cast<const T*>(v.p) + b * (n + 1) * v.ld_p;
  const float us = v.u_sample[b];

  if (warp == 0) {
    const int len = v.len != nullptr ? min(max(v.len[b], 0), n) : n;
    int a = len;
    for (int base = 0; base < len; base += 32) {
      const int i = base + lane;
      bool keep = true;
      if (i < len) {
        const int t = v.tokens[b * n + i];
        keep = t >= 0 && t < V;
        if (keep) keep = __fmul_rn(v.u_accept[b * n + i], to_f32(q0[i * v.ld_q + t])) < to_f32(p0[i * v.ld_p + t]);
      }
      const uint32_t refused = __ballot_sync(0xffffffffu, !keep);
      if (refused != 0u) {
        a = base + __ffs((int)refused) - 1;
        break;
      }
    }
    if (lane == 0) {
      s_a = a;
      s_len = len;
    }
  }
  __syncthreads();
  const int a = s_a;
  bool have_q = a < s_len;
  const Row<T, VEC> row = {p0 + a * v.ld_p, q0 + a * v.ld_q, V};

  // warp gw of the cluster's covers the contiguous elements [j0, j1)
  const int nw = (int)nrank * VW, gw = (int)rank * VW + warp;
  const int seg = ((V + nw - 1) / nw + row.CHUNK - 1) / row.CHUNK * row.CHUNK;
  const int j0 = (int)min((int64_t)gw * seg, (int64_t)V), j1 = min(j0 + seg, V);
  int drawn = -1;
  bool mine = false, empty = false;
  for (int pass = 0; pass < 2; ++pass) {
    long long sum = have_q ? row.template total<true>(j0, j1, lane) : row.template total<false>(j0, j1, lane);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_sum[pass][warp] = sum;
    if (nrank > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    long long total = 0, before = 0;
    for (int r = lane; r < nw; r += 32) {
      const long long s = nrank > 1 ? peer_ld64(smem_u32(&s_sum[pass][r % VW]), r / VW) : s_sum[pass][r];
      total += s;
      if (r < gw) before += s;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    if (total == 0) {
      if (!have_q) {
        empty = true;
        break;
      }
      have_q = false;   // p is nowhere above q: draw from p
      continue;
    }
    const long long un = min(max(__float2ll_rz(us * 16777216.f), 0ll), 16777215ll);
    const long long level = (total >> 24) * un + (((total & 16777215ll) * un) >> 24);
    if (before <= level && level < before + sum) {
      mine = true;
      drawn = have_q ? row.template find<true>(j0, j1, before, level, lane)
                     : row.template find<false>(j0, j1, before, level, lane);
    }
    break;
  }
  if (nrank > 1) cluster_arrive();   // this CTA has read its peers' sums; it waits for them at its end
  int32_t* out = v.out + b * (n + 1);
  if (rank == 0 && warp == 0) {
    for (int i = lane; i <= n; i += 32)
      if (i != a) out[i] = i < a ? v.tokens[b * n + i] : -1;
    if (lane == 0) {
      v.accepted[b] = a;
      if (empty) out[a] = -1;
    }
  }
  if (mine && lane == 0) out[a] = drawn;
  if (nrank > 1) cluster_wait();
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& v, int num_sms, cudaStream_t st) {
  // Clusters as large as keep every warp at work (8 elements a lane) until there are about three
  // CTAs for an SM (B = 128, V = 131072: 34 us by 4, 50 by one, 43 by 8; B = 16: 8.1 by 8, 14.4 by one).
  int c = 1;
  while (c < 8 && v.B * c * 2 <= 4 * num_sms && v.V > c * VT * 8) c *= 2;
  // 16-byte loads: rows that start and lie on whole vectors
  const int64_t w = v.dtype == MOE_F32 ? 4 : 8;
  const bool vec = v.ld_p % w == 0 && v.ld_q % w == 0;
  const dim3 grid((unsigned)(v.B * c));
  TraceScope ts(TP_VERIFY, st);
  if (v.dtype == MOE_F32)
    return vec ? launch_pdl(verify_kernel<float, true>, grid, VT, 0, c, st, v) : launch_pdl(verify_kernel<float, false>, grid, VT, 0, c, st, v);
  return vec ? launch_pdl(verify_kernel<__nv_bfloat16, true>, grid, VT, 0, c, st, v)
             : launch_pdl(verify_kernel<__nv_bfloat16, false>, grid, VT, 0, c, st, v);
}

}  // namespace moe
