// Layer norm of rows, with the residual's sum in front of it, and its gradients.
//
//   s = x (+ r),  mean = sum s / N,  var = sum (s - mean)^2 / N,  rstd = 1 / sqrt(var + eps)
//   y = (s - mean) rstd w (+ b)
//   u = dy w,  xh = (s - mean) rstd,  dx = rstd (u - mean(u) - xh mean(u xh)) (+ d_sum)
//   dw = sum_m dy xh,  db = sum_m dy
//
// A row stays in registers between its sums and its way out, so every operand is read once; the
// variance is that of the centred values (no difference of large numbers). All of it is bound by HBM.
#include "common.cuh"
#include "launch.cuh"
#include "ops.h"
#include "trace.h"

namespace moe {
namespace {

constexpr int kVecs = 4;   // vectors of 8 elements that a thread holds of a row

// Vector elements c .. c + 7 of a row, n of which exist. VEC: rows start on 16-byte boundaries.
template <typename T, bool VEC>
__device__ __forceinline__ void load_row(Vec8<T>& v, const T* row, int c, int n, const T* end) {
  if constexpr (VEC) {
    if (n >= 8) {
      v.load_plain(row + c);
    } else {
      T* e = reinterpret_cast<T*>(&v);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = i < n ? row[c + i] : T(0.f);
    }
  } else {
    load8_unaligned(v, row + c, end, n);
  }
}
template <typename T, bool VEC> __device__ __forceinline__ void store_row(const float* f, T* row, int c, int n) {
  if (VEC && n >= 8) {
    Vec8<T> v;
    v.from_float(f);
    v.store(row + c);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) row[c + i] = from_f32<T>(f[i]);
  }
}
// s = x (+ r) of a row's vector
template <typename T, bool VEC>
__device__ __forceinline__ void load_sum(float (&f)[8], const T* x, const T* r, int c, int n, const T* x_end, const T* r_end) {
  Vec8<T> v;
  load_row<T, VEC>(v, x, c, n, x_end);
  v.to_float(f);
  if (r != nullptr) {
    float g[8];
    load_row<T, VEC>(v, r, c, n, r_end);
    v.to_float(g);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += g[j];
  }
}
template <typename T> __device__ __forceinline__ const T* end_of(const void* p, int64_t M, int64_t ld, int N) {
  return static_cast<const T*>(p) + (M - 1) * ld + N;
}

// Sums of two values over the block, the same in every thread. `s`: 64 floats, not in use by an
// earlier call that a thread may still read (two buffers, taken in turn).
__device__ __forceinline__ float2 block_sums(float a, float b, float* s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if (nw == 1) return make_float2(a, b);
  if (lane == 0) {
    s[warp] = a;
    s[32 + warp] = b;
  }
  __syncthreads();
  a = lane < nw ? s[lane] : 0.f;
  b = lane < nw ? s[32 + lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  return make_float2(a, b);
}

template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormArgs a) {
  __shared__ float sums[2][64];
  pdl_start();
  pdl_wait();
  const int N = a.N;
  const int64_t m = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + m * a.ld_x;
  const T* r = a.res != nullptr ? static_cast<const T*>(a.res) + m * a.ld_res : nullptr;
  float f[kVecs][8];
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8, n = N - c;
    if (n > 0) {
      load_sum<T, VEC>(f[i], x, r, c, n, end_of<T>(a.x, a.M, a.ld_x, N), end_of<T>(a.res, a.M, a.ld_res, N));
      if (a.sum != nullptr) store_row<T, VEC>(f[i], static_cast<T*>(a.sum) + m * a.ld_sum, c, n);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j >= n) f[i][j] = 0.f;
        t += f[i][j];
      }
    }
  }
  const float mean = block_sums(t, 0.f, sums[0]).x * a.inv_n;
  t = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int n = N - (threadIdx.x + i * blockDim.x) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) {
        f[i][j] -= mean;
        t = fmaf(f[i][j], f[i][j], t);
      }
  }
  const float rstd = 1.f / sqrtf(block_sums(t, 0.f, sums[1]).x * a.inv_n + a.eps);
  if (threadIdx.x == 0 && a.stats != nullptr) reinterpret_cast<float2*>(a.stats)[m] = make_float2(mean, rstd);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8, n = N - c;
    if (n > 0) {
      float w[8], b[8];
      Vec8<W> v;
      load_row<W, true>(v, static_cast<const W*>(a.w), c, n, nullptr);
      v.to_float(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = 0.f;
      if (a.b != nullptr) {
        load_row<W, true>(v, static_cast<const W*>(a.b), c, n, nullptr);
        v.to_float(b);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] = fmaf(f[i][j] * rstd, w[j], b[j]);
      store_row<T, VEC>(f[i], static_cast<T*>(a.y) + m * a.ld_y, c, n);
    }
  }
}

template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(1024) norm_dx_kernel(const NormBwdArgs a) {
  __shared__ float sums[64];
  pdl_start();
  pdl_wait();
  const int N = a.N;
  const int64_t m = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + m * a.ld_x;
  const T* r = a.res != nullptr ? static_cast<const T*>(a.res) + m * a.ld_res : nullptr;
  const T* dy = static_cast<const T*>(a.dy) + m * a.ld_dy;
  const float2 st = reinterpret_cast<const float2*>(a.stats)[m];
  float u[kVecs][8], xh[kVecs][8];
  float t = 0.f, tx = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8, n = N - c;
    if (n > 0) {
      float w[8];
      Vec8<T> v;
      Vec8<W> vw;
      load_sum<T, VEC>(xh[i], x, r, c, n, end_of<T>(a.x, a.M, a.ld_x, N), end_of<T>(a.res, a.M, a.ld_res, N));
      load_row<T, VEC>(v, dy, c, n, end_of<T>(a.dy, a.M, a.ld_dy, N));
      v.to_float(u[i]);
      load_row<W, true>(vw, static_cast<const W*>(a.w), c, n, nullptr);
      vw.to_float(w);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) {
          xh[i][j] = (xh[i][j] - st.x) * st.y;
          u[i][j] *= w[j];
          t += u[i][j];
          tx = fmaf(u[i][j], xh[i][j], tx);
        }
    }
  }
  const float2 c12 = block_sums(t, tx, sums);
  const float c1 = c12.x * a.inv_n, c2 = c12.y * a.inv_n;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8, n = N - c;
    if (n > 0) {
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = 0.f;
      if (a.d_sum != nullptr) {
        Vec8<T> v;
        load_row<T, VEC>(v, static_cast<const T*>(a.d_sum) + m * a.ld_ds, c, n, end_of<T>(a.d_sum, a.M, a.ld_ds, N));
        v.to_float(g);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = fmaf(st.y, u[i][j] - c1 - xh[i][j] * c2, g[j]);
      store_row<T, VEC>(g, static_cast<T*>(a.dx) + m * a.ld_dx, c, n);
    }
  }
}

// Column sums: a block owns 32 vectors of columns and a share of the rows, 8 warps taking rows in turn.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormBwdArgs a, int64_t rows) {
  __shared__ float s[2][8][32][9];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, N = a.N, c = (blockIdx.x * 32 + lane) * 8, n = N - c;
  pdl_start();
  pdl_wait();
  float dw[8], db[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = db[j] = 0.f;
  const int64_t m0 = blockIdx.y * rows, m1 = m0 + rows < a.M ? m0 + rows : a.M;
  if (n > 0) {
    for (int64_t m = m0 + warp; m < m1; m += 8) {
      const float2 st = reinterpret_cast<const float2*>(a.stats)[m];
      Vec8<T> v;
      float x[8], g[8];
      load_sum<T, VEC>(x, static_cast<const T*>(a.x) + m * a.ld_x,
                       a.res != nullptr ? static_cast<const T*>(a.res) + m * a.ld_res : nullptr, c, n, end_of<T>(a.x, a.M, a.ld_x, N),
                       end_of<T>(a.res, a.M, a.ld_res, N));
      load_row<T, VEC>(v, static_cast<const T*>(a.dy) + m * a.ld_dy, c, n, end_of<T>(a.dy, a.M, a.ld_dy, N));
      v.to_float(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[j] = fmaf(g[j], (x[j] - st.x) * st.y, dw[j]);
        db[j] += g[j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s[0][warp][lane][j] = dw[j];
    s[1][warp][lane][j] = db[j];
  }
  __syncthreads();
  const int l = threadIdx.x >> 3, j = threadIdx.x & 7, at = (blockIdx.x * 32 + l) * 8 + j;
  if (at >= N) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += s[k][w][l][j];
    a.part[((int64_t)blockIdx.y * 2 + k) * N + at] = t;
  }
}

// dw and db from their partial sums, added in order.
template <typename W>
__global__ void __launch_bounds__(256) norm_join_kernel(const float* part, int n_part, int N, W* dw, W* db) {
  __shared__ float s[8][33];
  const int col = threadIdx.x & 31, r = threadIdx.x >> 5, n = blockIdx.x * 32 + col;
  W* out = blockIdx.y == 0 ? dw : db;
  pdl_start();
  pdl_wait();
  if (out == nullptr) return;
  float t = 0.f;
  if (n < N) {
#pragma unroll 4
    for (int i = r; i < n_part; i += 8) t += part[((int64_t)i * 2 + blockIdx.y) * N + n];
  }
  s[r][col] = t;
  __syncthreads();
  if (r == 0 && n < N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) t += s[i][col];
    out[n] = from_f32<W>(t);
  }
}

int norm_threads(int N) {
  const int t = ((N + 8 * kVecs - 1) / (8 * kVecs) + 31) & ~31;
  return t;
}

template <typename T, typename W> cudaError_t norm_fwd(const NormArgs& a, cudaStream_t st) {
  const bool vec = a.M == 1 || (a.ld_x % 8 == 0 && a.ld_y % 8 == 0 && (a.res == nullptr || a.ld_res % 8 == 0) &&
                                (a.sum == nullptr || a.ld_sum % 8 == 0));
  const dim3 grid((unsigned)a.M);
  return vec ? launch_pdl(norm_fwd_kernel<T, W, true>, grid, norm_threads(a.N), 0, 1, st, a)
             : launch_pdl(norm_fwd_kernel<T, W, false>, grid, norm_threads(a.N), 0, 1, st, a);
}

template <typename T, typename W> cudaError_t norm_bwd(const NormBwdArgs& a, cudaStream_t st) {
  const bool vec = a.M == 1 || (a.ld_x % 8 == 0 && a.ld_dy % 8 == 0 && (a.res == nullptr || a.ld_res % 8 == 0));
  // columns first: dx may be the buffer of an operand
  if (a.dw != nullptr || a.db != nullptr) {
    const int nx = (a.N + 255) / 256;
    int64_t rows = (a.M + kNormParts - 1) / kNormParts;
    if (rows < 8) rows = 8;
    const int parts = (int)((a.M + rows - 1) / rows);
    const cudaError_t e = vec ? launch_pdl(norm_columns_kernel<T, true>, dim3(nx, parts), 256, 0, 1, st, a, rows)
                              : launch_pdl(norm_columns_kernel<T, false>, dim3(nx, parts), 256, 0, 1, st, a, rows);
    if (e != cudaSuccess) return e;
    const cudaError_t j = launch_pdl(norm_join_kernel<W>, dim3((a.N + 31) / 32, 2), 256, 0, 1, st, (const float*)a.part, parts, a.N,
                                     static_cast<W*>(a.dw), static_cast<W*>(a.db));
    if (j != cudaSuccess) return j;
  }
  if (a.dx == nullptr) return cudaSuccess;
  const bool vdx = a.M == 1 || (vec && a.ld_dx % 8 == 0 && (a.d_sum == nullptr || a.ld_ds % 8 == 0));
  const dim3 grid((unsigned)a.M);
  return vdx ? launch_pdl(norm_dx_kernel<T, W, true>, grid, norm_threads(a.N), 0, 1, st, a)
             : launch_pdl(norm_dx_kernel<T, W, false>, grid, norm_threads(a.N), 0, 1, st, a);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, int dtype, int w_dtype, cudaStream_t st) {
  TraceScope ts(TP_NORM, st);
  if (dtype == MOE_F32) return norm_fwd<float, float>(a, st);
  return w_dtype == MOE_F32 ? norm_fwd<__nv_bfloat16, float>(a, st) : norm_fwd<__nv_bfloat16, __nv_bfloat16>(a, st);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, int w_dtype, cudaStream_t st) {
  TraceScope ts(TP_NORM_BWD, st);
  if (dtype == MOE_F32) return norm_bwd<float, float>(a, st);
  return w_dtype == MOE_F32 ? norm_bwd<__nv_bfloat16, float>(a, st) : norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, st);
}

}  // namespace moe
