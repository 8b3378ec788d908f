// The whole MoE layer for a few tokens in fp32, on the FMA pipes: the scores and the selection by the
// router's kernels, then one warp per hidden row and one per output row.
#include "common.cuh"
#include "ops.h"
#include "trace.h"

namespace moe {
namespace {

template <typename TA, typename TB>
__device__ __forceinline__ float warp_dot(const TA* __restrict__ a, const TB* __restrict__ b, int n, int lane) {
  float s = 0.f;
  for (int i = lane * 8; i < n; i += 256) {
    Vec8<TA> va;
    Vec8<TB> vb;
    float fa[8], fb[8];
    va.load(a + i);
    vb.load(b + i);
    va.to_float(fa);
    vb.to_float(fb);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(fa[j], fb[j], s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// blockIdx.y: token copy q < T*k, or T*k + s*T + t for shared expert s. One warp per hidden row.
template <typename T>
__global__ void __launch_bounds__(256) decode_hidden_kernel(const DecodeArgs a) {
  const moe_dims& D = a.dm;
  const int lane = threadIdx.x & 31, j = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t Tk = D.T * D.k, q = blockIdx.y;
  const bool sh = q >= Tk;
  const int f = sh ? D.f_s : D.f;
  if (j >= f) return;
  const int64_t t = sh ? (q - Tk) % D.T : q / D.k;
  const int e = sh ? (int)((q - Tk) / D.T) : reinterpret_cast<const int32_t*>(a.ws + a.L.idx)[q];
  const float w = sh ? 1.f : reinterpret_cast<const float*>(a.ws + a.L.gate)[q];
  const T* w13 = static_cast<const T*>(sh ? a.ws13 : a.w13) + (int64_t)e * 2 * f * D.d;
  const T* x = static_cast<const T*>(a.x) + t * D.d;
  const float g = warp_dot(w13 + (int64_t)j * D.d, x, D.d, lane);
  const float u = warp_dot(w13 + (int64_t)(f + j) * D.d, x, D.d, lane);
  float* h = reinterpret_cast<float*>(a.ws + (sh ? a.L.hs : a.L.h)) + (sh ? q - Tk : q) * f;
  if (lane == 0) h[j] = w * silu_f(g) * u;
}

// blockIdx.y: token. One warp per output row.
template <typename T>
__global__ void __launch_bounds__(256) decode_output_kernel(const DecodeArgs a) {
  const moe_dims& D = a.dm;
  const int lane = threadIdx.x & 31, n = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t t = blockIdx.y;
  if (n >= D.d) return;
  const float* h = reinterpret_cast<const float*>(a.ws + a.L.h);
  const float* hs = reinterpret_cast<const float*>(a.ws + a.L.hs);
  float y = 0.f;
  for (int j = 0; j < D.k; ++j) {
    const int64_t q = t * D.k + j;
    const int e = reinterpret_cast<const int32_t*>(a.ws + a.L.idx)[q];
    y += warp_dot(static_cast<const T*>(a.w2) + ((int64_t)e * D.d + n) * D.f, h + q * D.f, D.f, lane);
  }
  for (int s = 0; s < D.S; ++s)
    y += warp_dot(static_cast<const T*>(a.ws2) + ((int64_t)s * D.d + n) * D.f_s,
                  hs + (s * D.T + t) * D.f_s, D.f_s, lane);
  if (lane == 0) {
    if (a.residual != nullptr) y += to_f32(static_cast<const T*>(a.residual)[t * D.d + n]);
    static_cast<T*>(a.y)[t * D.d + n] = from_f32<T>(y);
  }
}

template <typename T>
cudaError_t run_ffn(const DecodeArgs& a, cudaStream_t st) {
  const moe_dims& D = a.dm;
  const int fm = D.S > 0 && D.f_s > D.f ? D.f_s : D.f;
  decode_hidden_kernel<T><<<dim3((fm + 7) / 8, (unsigned)(D.T * (D.k + D.S))), 256, 0, st>>>(a);
  decode_output_kernel<T><<<dim3((D.d + 7) / 8, (unsigned)D.T), 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

int launch_decode_simt(const DecodeArgs& a, int num_sms, cudaStream_t st) {
  const moe_dims& D = a.dm;
  float* logits = reinterpret_cast<float*>(a.ws + a.L.logits);
  int32_t* idx = reinterpret_cast<int32_t*>(a.ws + a.L.idx);
  float* gate = reinterpret_cast<float*>(a.ws + a.L.gate);
  int32_t* counts = reinterpret_cast<int32_t*>(a.ws + a.L.counts);
  if (a.logits_in == nullptr && launch_router_logits(a.x, a.w_r, D, logits, st) != cudaSuccess) return MOE_ERR_LAUNCH;
  if (cudaMemsetAsync(counts, 0, 4 * D.E, st) != cudaSuccess) return MOE_ERR_CUDA;
  if (launch_route_topk(a.logits_in != nullptr ? a.logits_in : logits, a.bias, D.T, D.E, D.k, idx, gate, counts,
                        num_sms, st) != cudaSuccess)
    return MOE_ERR_LAUNCH;
  const size_t n = 4 * (size_t)D.T * D.k;
  if (a.idx_out != nullptr && cudaMemcpyAsync(a.idx_out, idx, n, cudaMemcpyDeviceToDevice, st) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (a.gate_out != nullptr && cudaMemcpyAsync(a.gate_out, gate, n, cudaMemcpyDeviceToDevice, st) != cudaSuccess)
    return MOE_ERR_CUDA;
  TraceScope ts(TP_DECODE, st);
  const cudaError_t e = run_ffn<float>(a, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // namespace moe
