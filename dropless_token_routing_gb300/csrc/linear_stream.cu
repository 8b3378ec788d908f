// The linear layer's serving form: y = act(x W^T + b) + r for few rows, bf16, as one stream of W
// (stream.cuh). The result leaves the tensor memory transposed (lanes are outputs), so that each
// token's 128 outputs of a tile are contiguous.
#include <string.h>

#include <mutex>

#include "act.cuh"
#include "stream.cuh"
#include "trace.h"

namespace moe {
namespace {

using namespace stream;

struct LinearStream {
  CUtensorMap w, x;
  int M, N, nkb, tiles;
  const __nv_bfloat16 *bias, *res;
  __nv_bfloat16 *z, *y;
  int64_t ld_res, ld_y;
  bool vec;             // rows of y, res and z hold whole 16-byte vectors
  uint32_t* header;
  float* part;          // [CTA][NT][128]
};

template <int ACT> struct Finish {
  const LinearStream& g;
  __device__ void prepare(int64_t) {}
  // 8 outputs of one token per thread and step
  __device__ void finish(int64_t tile, int c0, const float* acc) {
    const int n0 = (int)tile * BM, tid = threadIdx.x - 64;
    const int q = (tid & 15) * 8, n = n0 + q;
    if (n >= g.N) return;
    const int cols = min(8, g.N - n);
    float b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = g.bias != nullptr && i < cols ? __bfloat162float(g.bias[n + i]) : 0.f;
    for (int c = tid >> 4; c < 64 && c0 + c < g.M; c += 16) {
      const int64_t m = c0 + c;
      float v[8], r[8];
      *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(acc + c * PITCH + q);
      *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(acc + c * PITCH + q + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] += b[i];
        r[i] = 0.f;
      }
      Vec8<__nv_bfloat16> p;
      if (g.vec) {
        if (g.res != nullptr) {
          p.v = *reinterpret_cast<const uint4*>(g.res + m * g.ld_res + n);   // may be y's own buffer
          p.to_float(r);
        }
        if (g.z != nullptr) {
          p.from_float(v);
          p.store(g.z + m * g.N + n);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act_f<ACT>(v[i]) + r[i];
        p.from_float(v);
        p.store(g.y + m * g.ld_y + n);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i >= cols) break;
          const float res = g.res != nullptr ? __bfloat162float(g.res[m * g.ld_res + n + i]) : 0.f;
          if (g.z != nullptr) g.z[m * g.N + n + i] = __float2bfloat16_rn(v[i]);
          g.y[m * g.ld_y + n + i] = __float2bfloat16_rn(act_f<ACT>(v[i]) + res);
        }
      }
    }
  }
};

template <int NT, int ACT>
__global__ void __launch_bounds__(THREADS, 1) linear_stream_kernel(const __grid_constant__ LinearStream g) {
  constexpr int STAGES = Cfg<NT>::stages(0);
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) Bars b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem_base = smem_u32(smem);
  float* acc = reinterpret_cast<float*>(smem + STAGES * Cfg<NT>::STAGE);
  int* err = reinterpret_cast<int*>(g.header);
  const int cta = (int)blockIdx.x, n_cta = (int)gridDim.x;
  setup<NT, STAGES>(b, warp);
  const uint32_t epoch = *reinterpret_cast<volatile uint32_t*>(g.header + 1) + 1;
  Run run(g.tiles, g.nkb, cta, n_cta);

  if (warp == 0) {
    if (lane == 0) {
      Ring<STAGES> ring;
      int64_t loaded = 0;
      bool ok = true;
      while (ok && run.next()) {
        const int n0 = (int)run.s.t * BM;
        for (int kb = run.s.k0; kb < run.s.k1; ++kb) {
          if (!mbar_wait_bounded(smem_u32(&b.empty[ring.stage]), ring.phase ^ 1u, &b.abort, err, kWaitLimitNs)) {
            ok = false;
            break;
          }
          const uint32_t a_s = smem_base + ring.stage * Cfg<NT>::STAGE, bar = smem_u32(&b.full[ring.stage]);
          mbar_arrive_expect_tx(bar, Cfg<NT>::STAGE);
          tma2d(a_s, &g.w, bar, kb * BK, n0);
          tma2d(a_s + A_BYTES, &g.x, bar, kb * BK, 0);
          ring.step();
          ++loaded;
        }
      }
      drain<STAGES>(b, ring, loaded, err);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      Ring<STAGES> ring;
      int it = 0;
      mma_run<NT, STAGES>(b, smem_base, run, ring, it, err);
      umma1_commit(smem_u32(&b.final));   // every MMA retired before the tensor memory is released
      mbar_wait_bounded(smem_u32(&b.final), 0, nullptr, err, kWaitLimitNs);
    }
    __syncwarp();
  } else {
    int it = 0;
    Finish<ACT> f{g};
    take_run<NT>(b, run, it, cta, g.header + 256, epoch, g.part, acc, err, f);
  }
  teardown<NT>(b, warp);
  leave(g.header, epoch);
}

template <int NT, int ACT>
int launch_nt(LinearStream& g, const GemmArgs& a, int num_sms, cudaStream_t st) {
  constexpr int SMEM = Cfg<NT>::smem(0);
  auto kernel = linear_stream_kernel<NT, ACT>;
  static std::mutex mu;   // the shared-memory attribute is set once per device
  static bool attr_set[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MOE_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!attr_set[dev]) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess) return MOE_ERR_CUDA;
      attr_set[dev] = true;
    }
  }
  if (!map2d_ld(&g.w, a.b, a.K, a.N, a.bn, BK, BM) || !map2d_ld(&g.x, a.a, a.K, a.M, a.am, BK, NT)) return MOE_ERR_CUDA;
  const int64_t units = (int64_t)g.tiles * g.nkb;
  int ctas = num_sms < kMaxStreamCtas ? num_sms : kMaxStreamCtas;
  if (units / kMinStreamRun < ctas) ctas = units < kMinStreamRun ? 1 : (int)(units / kMinStreamRun);
  TraceScope ts(TP_LINEAR, st);
  kernel<<<ctas, THREADS, SMEM, st>>>(g);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

template <int NT>
int launch_act(LinearStream& g, const GemmArgs& a, int num_sms, cudaStream_t st) {
#define MOE_S(A) return launch_nt<NT, A>(g, a, num_sms, st)
  MOE_ACT_SWITCH(a.act, MOE_S)
#undef MOE_S
  return MOE_OK;
}

}  // namespace

size_t linear_stream_part_bytes(int64_t M) {
  const int nt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
  return (size_t)kMaxStreamCtas * nt * BM * 4;
}

int launch_linear_stream(const GemmArgs& a, uint8_t* ws, size_t part, int num_sms, cudaStream_t st) {
  LinearStream g;
  memset(&g, 0, sizeof(g));
  g.M = (int)a.M;
  g.N = a.N;
  g.nkb = (int)((a.K + BK - 1) / BK);
  g.tiles = (a.N + BM - 1) / BM;
  g.bias = static_cast<const __nv_bfloat16*>(a.bias);
  g.res = static_cast<const __nv_bfloat16*>(a.res);
  g.z = static_cast<__nv_bfloat16*>(a.z_out);
  g.y = static_cast<__nv_bfloat16*>(a.c);
  g.ld_res = a.ld_res;
  g.ld_y = a.ldc;
  g.vec = a.N % 8 == 0 && a.ldc % 8 == 0 && (a.res == nullptr || a.ld_res % 8 == 0);
  g.header = reinterpret_cast<uint32_t*>(ws);
  g.part = reinterpret_cast<float*>(ws + part);
  if (a.M <= 16) return launch_act<16>(g, a, num_sms, st);
  if (a.M <= 32) return launch_act<32>(g, a, num_sms, st);
  if (a.M <= 64) return launch_act<64>(g, a, num_sms, st);
  if (a.M <= 128) return launch_act<128>(g, a, num_sms, st);
  return launch_act<256>(g, a, num_sms, st);
}

}  // namespace moe
