// The linear layer on the FMA pipes: products of any type, size, stride and alignment, and the
// elementwise half of its backward.
#include "act.cuh"
#include "ops.h"
#include "trace.h"

namespace moe {
namespace {

constexpr int GM = 64, GN = 64, GK = 16;

// One 64 x 64 tile of C = act(A B^T + bias) + res per block, 4 x 4 of it per thread. AK / BK:
// k is the contiguous index of A / B (else the row is), so that the tile loads coalesce.
template <typename T, int ACT, bool AK, bool BK>
__global__ void __launch_bounds__(256) gemm_simt_kernel(const GemmArgs g) {
  __shared__ float As[GK][GM + 4];
  __shared__ float Bs[GK][GN + 4];
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int64_t m0 = (int64_t)blockIdx.x * GM;
  const int n0 = blockIdx.y * GN;
  const T* A = static_cast<const T*>(g.a);
  const T* B = static_cast<const T*>(g.b);
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < g.K; k0 += GK) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = tid + 256 * i;
      const int ar = AK ? s / GK : s % GM, ac = AK ? s % GK : s / GM;
      const int br = BK ? s / GK : s % GN, bc = BK ? s % GK : s / GN;
      As[ac][ar] = m0 + ar < g.M && k0 + ac < g.K ? to_f32(A[(m0 + ar) * g.am + (k0 + ac) * g.ak]) : 0.f;
      Bs[bc][br] = n0 + br < g.N && k0 + bc < g.K ? to_f32(B[(n0 + br) * g.bn + (k0 + bc) * g.bk]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < GK; ++k) {
      const float4 a4 = *reinterpret_cast<const float4*>(&As[k][ty * 4]);
      const float4 b4 = *reinterpret_cast<const float4*>(&Bs[k][tx * 4]);
      const float av[4] = {a4.x, a4.y, a4.z, a4.w}, bv[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
    __syncthreads();
  }
  const T* bias = static_cast<const T*>(g.bias);
  const T* res = static_cast<const T*>(g.res);
  T* z = static_cast<T*>(g.z_out);
  T* c = static_cast<T*>(g.c);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty * 4 + i;
    if (m >= g.M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (n >= g.N) continue;
      const float v = acc[i][j] + (bias != nullptr ? to_f32(bias[n]) : 0.f);
      if (z != nullptr) z[m * g.N + n] = from_f32<T>(v);
      c[m * g.ldc + n] = from_f32<T>(act_f<ACT>(v) + (res != nullptr ? to_f32(res[m * g.ld_res + n]) : 0.f));
    }
  }
}

template <typename T, int ACT>
void gemm_simt(const GemmArgs& g, cudaStream_t st) {
  const dim3 grid((unsigned)((g.M + GM - 1) / GM), (unsigned)((g.N + GN - 1) / GN));
  if (g.ak == 1 && g.bk == 1) gemm_simt_kernel<T, ACT, true, true><<<grid, 256, 0, st>>>(g);
  else if (g.ak == 1) gemm_simt_kernel<T, ACT, true, false><<<grid, 256, 0, st>>>(g);
  else if (g.bk == 1) gemm_simt_kernel<T, ACT, false, true><<<grid, 256, 0, st>>>(g);
  else gemm_simt_kernel<T, ACT, false, false><<<grid, 256, 0, st>>>(g);
}

// dz = dy * act'(z), and its column sums. A block takes 256 columns and every gridDim.y-th group of
// 8 rows: 8 columns per lane, a row per warp. Its warps' sums are added in order into one row of
// `part` per block. (8-element vectors where the rows allow, else element by element.)
template <typename T, int ACT, bool VEC>
__global__ void __launch_bounds__(256) linear_dz_kernel(const T* __restrict__ dy, int64_t ld_dy,
                                                        const T* __restrict__ z, int64_t M, int N,
                                                        T* __restrict__ dz, int64_t ld_dz,
                                                        float* __restrict__ part) {
  __shared__ float s[8][256 + 8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = blockIdx.x * 256 + lane * 8, cols = min(8, N - n);
  float sum[8] = {};
  auto load = [&](const T* p, float (&v)[8]) {
    if (VEC) {
      Vec8<T> u;
      u.load(p);
      u.to_float(v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < cols ? to_f32(p[i]) : 0.f;
    }
  };
  if (cols > 0) {
#pragma unroll(ACT == MOE_ACT_NONE ? 8 : 4)
    for (int64_t m = (int64_t)blockIdx.y * 8 + warp; m < M; m += (int64_t)gridDim.y * 8) {
      float v[8], zv[8];
      load(dy + m * ld_dy + n, v);
      if constexpr (ACT != MOE_ACT_NONE) {
        load(z + m * N + n, zv);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= sizeof(T) == 2 ? act_slope_fast<ACT>(zv[i]) : act_slope<ACT>(zv[i]);
      }
      if (dz != nullptr) {
        T* out = dz + m * ld_dz + n;
        if (VEC) {
          Vec8<T> u;
          u.from_float(v);
          u.store(out);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < cols) out[i] = from_f32<T>(v[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += v[i];
    }
  }
  if (part == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) s[warp][lane * 8 + i] = sum[i];
  __syncthreads();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c < N) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += s[w][threadIdx.x];
    part[(int64_t)blockIdx.y * N + c] = t;
  }
}

// db = the sum of n_part rows: 32 columns per block, 8 threads each, added in order.
template <typename T>
__global__ void __launch_bounds__(256) linear_db_kernel(const float* __restrict__ part, int n_part, int N, T* __restrict__ db) {
  __shared__ float s[8][33];
  const int col = threadIdx.x & 31, r = threadIdx.x >> 5, n = blockIdx.x * 32 + col;
  float t = 0.f;
  if (n < N) {
#pragma unroll 8
    for (int i = r; i < n_part; i += 8) t += part[(int64_t)i * N + n];
  }
  s[r][col] = t;
  __syncthreads();
  if (r == 0 && n < N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) t += s[i][col];
    db[n] = from_f32<T>(t);
  }
}

template <typename T>
cudaError_t linear_dz(const void* dy, int64_t ld_dy, const void* z, int act, int64_t M, int N, void* dz,
                      int64_t ld_dz, float* part, void* db, cudaStream_t st) {
  // about 1200 blocks (8 on an SM), of at least 32 rows
  const int nx = (N + 255) / 256;
  int64_t split = (1216 + nx - 1) / nx;
  if (split > (M + 31) / 32) split = (M + 31) / 32;
  if (split > kDbSplit) split = kDbSplit;
  const dim3 grid(nx, (unsigned)split);
  const bool vec = N % 8 == 0 && ld_dy % 8 == 0;   // ld_dz is a multiple of 8
  const T *dyp = static_cast<const T*>(dy), *zp = static_cast<const T*>(z);
  T* dzp = static_cast<T*>(dz);
  float* pp = db != nullptr ? part : nullptr;
#define MOE_DZ(A)                                                                                   \
  if (vec) linear_dz_kernel<T, A, true><<<grid, 256, 0, st>>>(dyp, ld_dy, zp, M, N, dzp, ld_dz, pp); \
  else linear_dz_kernel<T, A, false><<<grid, 256, 0, st>>>(dyp, ld_dy, zp, M, N, dzp, ld_dz, pp)
  MOE_ACT_SWITCH(act, MOE_DZ)
#undef MOE_DZ
  if (db != nullptr) linear_db_kernel<T><<<(N + 31) / 32, 256, 0, st>>>(part, (int)split, N, static_cast<T*>(db));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gemm_simt(const GemmArgs& g, cudaStream_t st) {
  TraceScope ts(TP_LINEAR, st);
  if (g.dtype == MOE_F32) {
#define MOE_G(A) gemm_simt<float, A>(g, st)
    MOE_ACT_SWITCH(g.act, MOE_G)
#undef MOE_G
  } else {
#define MOE_G(A) gemm_simt<__nv_bfloat16, A>(g, st)
    MOE_ACT_SWITCH(g.act, MOE_G)
#undef MOE_G
  }
  return cudaGetLastError();
}

cudaError_t launch_linear_dz(const void* dy, int64_t ld_dy, const void* z, int act, int64_t M, int N, int dtype,
                             void* dz, int64_t ld_dz, float* db_part, void* db, cudaStream_t st) {
  TraceScope ts(TP_LINEAR_DZ, st);
  return dtype == MOE_F32 ? linear_dz<float>(dy, ld_dy, z, act, M, N, dz, ld_dz, db_part, db, st)
                          : linear_dz<__nv_bfloat16>(dy, ld_dy, z, act, M, N, dz, ld_dz, db_part, db, st);
}

}  // namespace moe
