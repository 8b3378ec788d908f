// The linear layer's serving form: y = act(x W^T + b) + r for few rows, bf16, as one stream of W
// (stream.cuh). The result leaves the tensor memory transposed (lanes are outputs), so that each
// token's outputs of a tile are contiguous.
//
// W's rows are divided evenly: a cluster of 1, 2, 4 or 8 CTAs takes tiles of R <= 128 rows, R such
// that all clusters have the same number of tiles, and its CTAs each a share of K. They join their
// sums through distributed shared memory, each CTA finishing a share of the token columns: a
// join through global memory costs fences, flags and loads of about 2 us each behind the stream.
// The host picks the cluster size with the least time for a CTA's share (launch_nt).
//
// z and y are rounded to bf16 from the fp32 sum, each once. Bound by HBM for large W, by the launch
// and the join (5 us together) for small ones: M = 16, 7680 x 7680: 22.5 us, 5.3 TB/s; M = 37, N =
// 4097, K = 7168: 15.4 us, 3.9 TB/s; M = 1, N = 7680, K = 2048: 8.6 us, 3.6 TB/s; M = 1, 1000 x 512:
// 3.8 us.
#include <string.h>

#include <mutex>

#include "act.cuh"
#include "launch.cuh"
#include "stream.cuh"
#include "trace.h"

namespace moe {
namespace {

using namespace stream;

struct LinearStream {
  CUtensorMap w, x;
  int M, N, nkb, tiles, rows;   // rows of W in a tile
  int act;
  const __nv_bfloat16 *bias, *res;
  __nv_bfloat16 *z, *y;
  int64_t ld_res, ld_y, ld_z;
  bool vec;             // rows of y and res hold whole 16-byte vectors (z's and tiles do)
  int* err;
};

__device__ __forceinline__ float4 peer_ld4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float peer_ld1(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
// One arrival on this barrier of every CTA of the cluster.
__device__ __forceinline__ void arrive_all(uint64_t* bar, int cluster) {
  for (int i = 0; i < cluster; ++i)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer_addr(smem_u32(bar), i)) : "memory");
}
// The wait for the other CTAs' arrivals (their shared memory may be read, or written over, after).
static __device__ __noinline__ bool peers_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  const uint64_t t0 = global_ns();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (*abort) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      record_error(err, MOE_ERR_DEVICE_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
}

// 8 outputs (n .. n + 7) of token m.
__device__ __forceinline__ void finish8(const LinearStream& g, float (&v)[8], const float (&b)[8], int64_t m, int n) {
  float r[8] = {};
  Vec8<__nv_bfloat16> p;
  if (g.res != nullptr) {
    p.v = *reinterpret_cast<const uint4*>(g.res + m * g.ld_res + n);   // may be y's own buffer
    p.to_float(r);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += b[i];
  if (g.z != nullptr) {
    p.from_float(v);
    p.store(g.z + m * g.ld_z + n);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = act_any_fast(g.act, v[i]) + r[i];
  p.from_float(v);
  p.store(g.y + m * g.ld_y + n);
}

template <int NT>
__global__ void __launch_bounds__(THREADS, 1) linear_stream_kernel(const __grid_constant__ LinearStream g) {
  constexpr int STAGES = Cfg<NT>::stages(0), STAGE = Cfg<NT>::STAGE;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) Bars b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem_base = smem_u32(smem);
  float* acc = reinterpret_cast<float*>(smem + STAGES * STAGE);
  uint32_t cl, rank;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(cl));
  rank = cluster_rank();
  const int tile0 = (int)cluster_id(), step = (int)cluster_count();
  const int k0 = (int)((int64_t)g.nkb * rank / cl), k1 = (int)((int64_t)g.nkb * (rank + 1) / cl);
  pdl_start();
  setup<NT, STAGES>(b, warp, (int)cl);
  if (cl > 1) cluster_sync_all();   // the peers' barriers are initialised before any arrival
  pdl_wait();

  if (warp == 0) {
    // the whole warp, one lane issuing (see tc_common.cuh)
    const bool one = elect_one();
    Ring<STAGES> ring;
    int64_t loaded = 0;
    bool ok = true;
    const uint32_t bytes = (uint32_t)(g.rows + NT) * BK * 2;
    for (int tile = tile0; ok && tile < g.tiles; tile += step) {
      const int n0 = tile * g.rows;   // rows past the tile keep what was in the stage
      for (int kb = k0; kb < k1; ++kb) {
        ok = warp_bar_wait(smem_u32(&b.empty[ring.stage]), ring.phase ^ 1u, &b.abort, g.err);
        if (!ok) break;
        if (one) {
          const uint32_t a_s = smem_base + ring.stage * STAGE, bar = smem_u32(&b.full[ring.stage]);
          mbar_arrive_expect_tx(bar, bytes);
          tma2d(a_s, &g.w, bar, kb * BK, n0);
          tma2d(a_s + A_BYTES, &g.x, bar, kb * BK, 0);
        }
        ring.step();
        ++loaded;
      }
    }
    if (one) drain<STAGES>(b, ring, loaded, g.err);
    __syncwarp();
  } else if (warp == 1) {
    Ring<STAGES> ring;
    int it = 0;
    const bool one = elect_one();
    for (int tile = tile0; tile < g.tiles; tile += step, ++it)
      if (!mma_tile<NT, STAGES>(b, smem_base, k1 - k0, ring, it, one, g.err)) break;
    if (one) {
      umma1_commit(smem_u32(&b.final));   // every MMA retired before the tensor memory is released
      bar_wait(&b.final, 0, nullptr, g.err);
    }
    __syncwarp();
  } else {
    constexpr int HALF = NT / 2;
    const int lg = warp & 3, row = lg * 32 + lane, col0 = ((warp - 2) >> 2) * HALF, tid = threadIdx.x - 64;
    const int q = (tid & 15) * 8;   // this thread's 8 rows of W in a tile
    uint32_t parity = 0;
    bool ok = true;
    for (int tile = tile0, it = 0; ok && tile < g.tiles; tile += step, ++it) {
      const int buf = it & 1, n0 = tile * g.rows;
      // this thread's outputs: n0 + q .. + 7 where rows hold whole vectors, else n0 + lane + 32 i
      const int cols = min(g.rows, g.N - n0);
      float bias[8] = {};
      if (g.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int at = g.vec ? q + i : lane + 32 * i;
          if (at < cols && (g.vec || i < 4)) bias[i] = __bfloat162float(g.bias[n0 + at]);
        }
      }
      ok = bar_wait(&b.tfull[buf], (it >> 1) & 1, &b.abort, g.err);
      if (ct_any(!ok)) break;
      __syncwarp();
      tc_fence_after();
      const uint32_t t_base = b.tmem + ((uint32_t)(lg * 32) << 16) + (uint32_t)(buf * NT);
#pragma unroll
      for (int c = 0; c < HALF; c += 8) {
        uint32_t u[8];
        tmem_ld8(t_base + col0 + c, u);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[(col0 + c + i) * PITCH + row] = __uint_as_float(u[i]);
      }
      // this CTA's share of the tokens
      const int c_lo = g.M * (int)rank / (int)cl, c_hi = g.M * ((int)rank + 1) / (int)cl;
      ct_sync();
      if (cl > 1) {
        if (tid == 0) arrive_all(&b.peers_ready, (int)cl);
        ok = !ct_any(!peers_wait(&b.peers_ready, parity, &b.abort, g.err));
        if (!ok) break;
      }
      if (g.vec) {
        for (int c = c_lo + (tid >> 4); c < c_hi; c += 16) {
          float v[8] = {};
          for (uint32_t r0 = 0; r0 < cl; r0 += 4) {   // in the order of the ranks, four in flight
            float4 w[4][2];
#pragma unroll
            for (uint32_t r = 0; r < 4; ++r) {
              if (r0 + r >= cl) break;
              const uint32_t at = peer_addr(smem_u32(acc + c * PITCH + q), r0 + r);
              w[r][0] = peer_ld4(at);
              w[r][1] = peer_ld4(at + 16);
            }
#pragma unroll
            for (uint32_t r = 0; r < 4; ++r) {
              if (r0 + r >= cl) break;
              v[0] += w[r][0].x; v[1] += w[r][0].y; v[2] += w[r][0].z; v[3] += w[r][0].w;
              v[4] += w[r][1].x; v[5] += w[r][1].y; v[6] += w[r][1].z; v[7] += w[r][1].w;
            }
          }
          if (q < cols) finish8(g, v, bias, c, n0 + q);
        }
      } else {   // a token per warp, so that single elements still make whole sectors
        for (int c = c_lo + warp - 2; c < c_hi; c += CW) {
          const int64_t m = c;
          float v[4] = {}, res[4] = {};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (g.res != nullptr && lane + 32 * i < cols) res[i] = __bfloat162float(g.res[m * g.ld_res + n0 + lane + 32 * i]);
          for (uint32_t r0 = 0; r0 < cl; r0 += 4) {
            float w[4][4];
#pragma unroll
            for (uint32_t r = 0; r < 4; ++r) {
              if (r0 + r >= cl) break;
              const uint32_t at = peer_addr(smem_u32(acc + c * PITCH + lane), r0 + r);
#pragma unroll
              for (int i = 0; i < 4; ++i) w[r][i] = peer_ld1(at + 128 * i);
            }
#pragma unroll
            for (uint32_t r = 0; r < 4; ++r) {
              if (r0 + r >= cl) break;
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] += w[r][i];
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = lane + 32 * i;
            if (at >= cols) break;
            const float z = v[i] + bias[i];
            if (g.z != nullptr) g.z[m * g.ld_z + n0 + at] = __float2bfloat16_rn(z);
            g.y[m * g.ld_y + n0 + at] = __float2bfloat16_rn(act_any_fast(g.act, z) + res[i]);
          }
        }
      }
      ct_sync();
      // the peers have read this CTA's sums before they are written over (the last ones are not)
      if (cl > 1 && tile + step < g.tiles) {
        if (tid == 0) arrive_all(&b.peers_done, (int)cl);
        ok = !ct_any(!peers_wait(&b.peers_done, parity, &b.abort, g.err));
        if (!ok) break;
        parity ^= 1u;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&b.tempty[buf]));
    }
  }
  teardown<NT>(b, warp);
  if (cl > 1) cluster_sync_all();   // no CTA leaves while a peer may still reach its shared memory
}

// Clusters of `c` CTAs that can be resident at once (c = 1: the SMs).
template <int NT>
int resident(int c, int num_sms) {
  constexpr int SMEM = Cfg<NT>::smem(0);
  auto kernel = linear_stream_kernel<NT>;
  static std::mutex mu;   // per device, once: the shared-memory attribute and the counts
  static int count[kMaxDevices][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  const int i = c == 1 ? 0 : c == 2 ? 1 : c == 4 ? 2 : 3;
  std::lock_guard<std::mutex> lk(mu);
  if (count[dev][0] == 0) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess) return 0;
    count[dev][0] = num_sms;
  }
  if (count[dev][i] == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_sms / c * c));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = c;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) return 0;
    count[dev][i] = n;
  }
  return count[dev][i];
}

template <int NT>
int launch_nt(LinearStream& g, const GemmArgs& a, int num_sms, cudaStream_t st) {
  // The cluster size with the least time for a CTA, in bytes of its share of the stream (45 a ns): a K
  // block takes as long as kBlock bytes at least (0.16 us), a join as long as kJoin (1.7 us).
  // M = 8, 2048 x 2048: 6.4 us by 8 CTAs, 8.1 by one; M = 1, N = 7680, K = 2048: 9.5 by 2, 8.9 by one.
  constexpr int64_t kBlock = 7 << 10, kJoin = 76 << 10;
  int best = 0, best_rows = 0, best_tiles = 0, best_clusters = 0;
  int64_t best_cost = 0;
  for (int c = 1; c <= 8; c *= 2) {
    if (c > 1 && g.nkb / c < 4) break;
    const int ncl = resident<NT>(c, num_sms);
    if (ncl == 0) return MOE_ERR_CUDA;
    const int per = (g.N + ncl * BM - 1) / (ncl * BM);           // tiles of a cluster
    int rows = (g.N + ncl * per - 1) / (ncl * per);
    rows = (rows + 7) & ~7;                                      // whole vectors of outputs
    const int tiles = (g.N + rows - 1) / rows;
    const int64_t block = (int64_t)(rows + NT) * BK * 2;
    const int64_t cost = per * ((g.nkb + c - 1) / c * (block > kBlock ? block : kBlock) + (c > 1 ? kJoin : 0));
    if (best == 0 || cost < best_cost) {
      best = c;
      best_cost = cost;
      best_rows = rows;
      best_tiles = tiles;
      best_clusters = ncl < tiles ? ncl : tiles;
    }
  }
  g.rows = best_rows;
  g.tiles = best_tiles;
  if (!map2d_ld(&g.w, a.b, a.K, a.N, a.bn, BK, best_rows) || !map2d_ld(&g.x, a.a, a.K, a.M, a.am, BK, NT)) return MOE_ERR_CUDA;
  TraceScope ts(TP_LINEAR, st);
  return launch_pdl(linear_stream_kernel<NT>, dim3((unsigned)(best_clusters * best)), THREADS, Cfg<NT>::smem(0), best, st, g) ==
                 cudaSuccess
             ? MOE_OK
             : MOE_ERR_LAUNCH;
}

}  // namespace

int launch_linear_stream(const GemmArgs& a, uint8_t* ws, int num_sms, cudaStream_t st) {
  LinearStream g;
  memset(&g, 0, sizeof(g));
  g.M = (int)a.M;
  g.N = a.N;
  g.nkb = (int)((a.K + BK - 1) / BK);
  g.act = a.act;
  g.bias = static_cast<const __nv_bfloat16*>(a.bias);
  g.res = static_cast<const __nv_bfloat16*>(a.res);
  g.z = static_cast<__nv_bfloat16*>(a.z_out);
  g.y = static_cast<__nv_bfloat16*>(a.c);
  g.ld_res = a.ld_res;
  g.ld_y = a.ldc;
  g.ld_z = a.ld_z;
  g.vec = a.N % 8 == 0 && a.ldc % 8 == 0 && (a.res == nullptr || a.ld_res % 8 == 0);
  g.err = reinterpret_cast<int*>(ws);
  if (a.M <= 16) return launch_nt<16>(g, a, num_sms, st);
  if (a.M <= 32) return launch_nt<32>(g, a, num_sms, st);
  if (a.M <= 64) return launch_nt<64>(g, a, num_sms, st);
  return launch_nt<128>(g, a, num_sms, st);
}

}  // namespace moe
