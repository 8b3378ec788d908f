// Verification of drafted tokens: which of them stay, and the token drawn after the last one
// that stays.
//
// Only one row of the target's probabilities (and one of the draft's) is read per sequence: the
// row at the first refusal, or the one after the last kept token. Its weights are whole
// multiples of 2^-40 and are summed as 64-bit integers, so the sums, and with them the drawn
// token, do not depend on how the row is split over threads and CTAs.
#include "common.cuh"
#include "ops.h"
#include "trace.h"

namespace moe {
namespace {

constexpr int VT = 512, VW = VT / 32;   // threads and warps per CTA

__device__ __forceinline__ uint32_t ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The 64-bit word at shared address `a` of CTA `rank` of the cluster.
__device__ __forceinline__ long long peer_ld64(uint32_t a, uint32_t rank) {
  uint32_t p;
  long long v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(p) : "memory");
  return v;
}

// fp32 weight -> multiples of 2^-40; fmaxf takes NaN to 0, and the scaling is exact.
__device__ __forceinline__ long long mass(float r) {
  return __float2ll_rz(fminf(fmaxf(r, 0.f), 1.f) * 1099511627776.f);
}

template <typename T>
__device__ __forceinline__ long long weight(const T* p, const T* q, int64_t j) {
  const float pv = to_f32(p[j]);
  return mass(q != nullptr ? pv - to_f32(q[j]) : pv);
}

template <typename T>
__global__ void __launch_bounds__(VT) verify_kernel(const VerifyArgs v) {
  __shared__ int s_a, s_len;
  __shared__ long long s_sum[VW];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ctarank(), nrank = nctarank();
  const int64_t b = blockIdx.x / nrank;
  const int n = v.n, V = v.V;
  const T* q0 = static_cast<const T*>(v.q) + b * n * v.ld_q;
  const T* p0 = static_cast<const T*>(v.p) + b * (n + 1) * v.ld_p;

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
  const T* p = p0 + a * v.ld_p;
  const T* q = a < s_len ? q0 + a * v.ld_q : nullptr;

  // warp gw of the cluster's covers the contiguous elements [j0, j1)
  const int nw = (int)nrank * VW, gw = (int)rank * VW + warp;
  const int seg = ((V + nw - 1) / nw + 31) & ~31;
  const int j0 = min(gw * seg, V), j1 = min(j0 + seg, V);
  int drawn = -1;
  bool mine = false, empty = false;
  for (int pass = 0; pass < 2; ++pass) {
    long long sum = 0;
#pragma unroll 8
    for (int j = j0 + lane; j < j1; j += 32) sum += weight(p, q, j);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_sum[warp] = sum;
    cluster_sync();
    long long total = 0, before = 0;
    for (int r = lane; r < nw; r += 32) {
      const long long s = peer_ld64(smem_u32(&s_sum[r % VW]), r / VW);
      total += s;
      if (r < gw) before += s;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    cluster_sync();   // every CTA has read the sums before they are written again or freed
    if (total == 0) {
      if (q == nullptr) {
        empty = true;
        break;
      }
      q = nullptr;    // p is nowhere above q: draw from p
      continue;
    }
    const long long un = min(max(__float2ll_rz(v.u_sample[b] * 16777216.f), 0ll), 16777215ll);
    const long long level = (total >> 24) * un + (((total & 16777215ll) * un) >> 24);
    if (before <= level && level < before + sum) {
      mine = true;
      long long cum = before;
      for (int j = j0; j < j1; j += 32) {
        const long long w = j + lane < j1 ? weight(p, q, j + lane) : 0;
        long long c = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long t = __shfl_up_sync(0xffffffffu, c, o);
          if (lane >= o) c += t;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, cum + c > level);
        if (hit != 0u) {
          drawn = j + __ffs((int)hit) - 1;
          break;
        }
        cum += __shfl_sync(0xffffffffu, c, 31);
      }
    }
    break;
  }
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
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& v, int num_sms, cudaStream_t st) {
  int c = 1;
  while (c < 8 && v.B * c * 2 <= 2 * num_sms && v.V > c * VT * 8) c *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(v.B * c));
  cfg.blockDim = dim3(VT);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  TraceScope ts(TP_VERIFY, st);
  return v.dtype == MOE_F32 ? cudaLaunchKernelEx(&cfg, verify_kernel<float>, v)
                            : cudaLaunchKernelEx(&cfg, verify_kernel<__nv_bfloat16>, v);
}

}  // namespace moe
