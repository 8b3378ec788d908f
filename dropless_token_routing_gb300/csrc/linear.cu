// The linear layer's fp32 products, on the FMA pipes, and the elementwise half of its backward.
//
// The tensor cores have no fp32 type, and three bf16 parts would lose what fp32 keeps at the ends of
// its range. The products are bound by latency that 16 warps on an SM do not hide (ncu, 2048 x 2048 x
// 512: FMA pipe 55 % busy while a block runs, issue slots 39 %; a warp waits for fixed latencies, shared
// and global memory and instructions, with a block-wide barrier for every 16 of K): 1024 x 1024 x
// 1024: 51 us, 42 TFLOP/s; 900 x 900 x 4000: 162 us, 40 TFLOP/s (75 is the pipes' rate).
#include "act.cuh"
#include "launch.cuh"
#include "ops.h"
#include "trace.h"

namespace moe {
namespace {

constexpr int GM = 128, GN = 64, GK = 16, GT = 128;

// bias, z, activation, residual of one element and its way out.
__device__ __forceinline__ void finish_element(const GemmArgs& g, int64_t m, int n, float v) {
  if (g.bias != nullptr) v += static_cast<const float*>(g.bias)[n];
  if (g.z_out != nullptr) static_cast<float*>(g.z_out)[m * g.ld_z + n] = v;
  v = act_any(g.act, v);
  if (g.res != nullptr) v += static_cast<const float*>(g.res)[m * g.ld_res + n];
  static_cast<float*>(g.c)[m * g.ldc + n] = v;
}

// Two fp32 FMAs in one instruction (1024 x 1024 x 1024: 63 us, 68 with single ones).
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void fma_pair(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}

// A thread's share of an R x 16 operand tile: single elements, which any stride and alignment
// allows. KC: k is the contiguous index (16 lanes along k, rows 8 apart), else the row is (64 lanes
// along the rows, k two apart).
template <bool KC, int R> struct Operand {
  static constexpr int N = R * GK / GT, H = R / 64;   // elements; rows of a lane where rows are contiguous
  const float* p;      // this thread's first element at the present k
  int64_t rs, ks;
  int row0, k;         // its first row in the tile, its first k in the block
  int rows;            // rows of the tile that exist
  __device__ Operand(const void* base, int64_t row, int64_t k0, int64_t rs_, int64_t ks_, int64_t total, int tid) {
    row0 = KC ? tid / GK : tid % 64;
    k = KC ? tid % GK : tid / 64;
    rows = (int)(total - row < R ? total - row : R);
    rs = rs_;
    ks = ks_;
    p = static_cast<const float*>(base) + (row + row0) * rs + (k0 + k) * ks;
  }
  __device__ __forceinline__ static int row_of(int i) { return KC ? 8 * i : i % H * 64; }
  __device__ __forceinline__ static int k_of(int i) { return KC ? 0 : i / H * 2; }
  // left: k's of this block that exist
  __device__ __forceinline__ void load(float (&r)[N], int64_t left) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool in = row0 + row_of(i) < rows && k + k_of(i) < left;
      r[i] = in ? p[row_of(i) * rs + k_of(i) * ks] : 0.f;
    }
    p += GK * ks;
  }
  __device__ __forceinline__ void stage(float (*s)[R + 4], const float (&r)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) s[k + k_of(i)][row0 + row_of(i)] = r[i];
  }
};

// One 128 x 64 tile of A B^T per block (or a share of its K: blockIdx.z of gridDim.z, into `part`, whole
// tiles of fp32 sums), 8 x 8 of it per thread in quarters of 4 x 4: 4 shared-memory vectors per 64 FMAs
// (with 8 x 4 the shared memory was the limit). The next 16 of K are loaded into registers while
// the present ones are multiplied.
// Four blocks fit on an SM; the gradients' forms need the limit for that (2048 x 2048 x 512: dw 91.8 us,
// 96.7 with 154 registers), the forward one is there by itself.
template <bool AK, bool BK, bool SPLIT>
__global__ void __launch_bounds__(GT, BK ? 0 : 4) gemm_simt_kernel(const GemmArgs g, float* part) {
  __shared__ __align__(16) float As[2][GK][GM + 4];
  __shared__ __align__(16) float Bs[2][GK][GN + 4];
  const int tid = threadIdx.x, ty = tid >> 3, tx = tid & 7;
  pdl_wait();
  const int64_t m0 = (int64_t)blockIdx.x * GM;
  const int n0 = blockIdx.y * GN;
  int64_t k_lo = 0, k_hi = g.K;
  if (SPLIT) {
    const int64_t per = ((g.K + gridDim.z - 1) / gridDim.z + GK - 1) / GK * GK;
    k_lo = per * blockIdx.z < g.K ? per * blockIdx.z : g.K;
    k_hi = k_lo + per < g.K ? k_lo + per : g.K;
  }
  Operand<AK, GM> A(g.a, m0, k_lo, g.am, g.ak, g.M, tid);
  Operand<BK, GN> B(g.b, n0, k_lo, g.bn, g.bk, g.N, tid);
  float ra[A.N], rb[B.N];
  uint64_t acc[8][4] = {};   // pairs of columns
  A.load(ra, k_hi - k_lo);
  B.load(rb, k_hi - k_lo);
  A.stage(As[0], ra);
  B.stage(Bs[0], rb);
  __syncthreads();
  int buf = 0;
  for (int64_t k0 = k_lo; k0 < k_hi; k0 += GK, buf ^= 1) {
    const int64_t left = k_hi - k0 - GK;
    if (left > 0) {
      A.load(ra, left);
      B.load(rb, left);
    }
#pragma unroll
    for (int k = 0; k < GK; ++k) {
      float av[8];
      alignas(16) float bv[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        *reinterpret_cast<float4*>(av + 4 * h) = *reinterpret_cast<const float4*>(&As[buf][k][64 * h + ty * 4]);
        *reinterpret_cast<float4*>(bv + 4 * h) = *reinterpret_cast<const float4*>(&Bs[buf][k][32 * h + tx * 4]);
      }
      const uint64_t* b2 = reinterpret_cast<const uint64_t*>(bv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t a2 = pair_of(av[i], av[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) fma_pair(acc[i][j], a2, b2[j]);
      }
    }
    if (left > 0) {   // the other buffer was last read before the previous barrier
      A.stage(As[buf ^ 1], ra);
      B.stage(Bs[buf ^ 1], rb);
      __syncthreads();
    }
  }
  if (SPLIT) {
    float* out = part + (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * gridDim.z + blockIdx.z) * (GM * GN);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<ulonglong2*>(out + (i / 4 * 64 + ty * 4 + i % 4) * GN + h * 32 + tx * 4) =
            make_ulonglong2(acc[i][2 * h], acc[i][2 * h + 1]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t m = m0 + i / 4 * 64 + ty * 4 + i % 4;
    if (m >= g.M) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int n = n0 + j / 4 * 32 + tx * 4 + j % 4;
      if (n >= g.N) continue;
      finish_element(g, m, n, __uint_as_float((uint32_t)(acc[i][j / 2] >> (j % 2 * 32))));
    }
  }
}

// The shares of a divided K, added in order: a tile's row per warp. (Neither this kernel nor the product
// lets the next one start early: its blocks would then fill the SMs that are free first, several on
// one. 256 x 256 x 1024: 8.0 us, 16.4 if this one does.)
constexpr int JR = 8;   // rows of a block
__global__ void __launch_bounds__(32 * JR) gemm_join_kernel(const GemmArgs g, const float* part, int split) {
  const int lane = threadIdx.x & 31, r = blockIdx.z * JR + (threadIdx.x >> 5);
  const int64_t m = (int64_t)blockIdx.x * GM + r;
  const int n = blockIdx.y * GN + lane;
  const float* in = part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * split * (GM * GN) + r * GN + lane;
  pdl_wait();
  if (m >= g.M) return;
  float v[2] = {};
  for (int s0 = 0; s0 < split; s0 += 16) {   // 16 shares in flight
    float w[16][2];
#pragma unroll
    for (int s = 0; s < 16; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) w[s][h] = s0 + s < split ? __ldcg(in + (s0 + s) * (GM * GN) + 32 * h) : 0.f;
#pragma unroll
    for (int s = 0; s < 16; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) v[h] += w[s][h];
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (n + 32 * h < g.N) finish_element(g, m, n + 32 * h, v[h]);
}

// The layouts of the layer's products: forward (both operands along k), dX, dW.
template <bool SPLIT>
void gemm_layouts(const GemmArgs& g, float* part, const dim3& grid, cudaStream_t st) {
  if (g.ak == 1 && g.bk == 1) launch_pdl(gemm_simt_kernel<true, true, SPLIT>, grid, GT, 0, 1, st, g, part);
  else if (g.ak == 1) launch_pdl(gemm_simt_kernel<true, false, SPLIT>, grid, GT, 0, 1, st, g, part);
  else launch_pdl(gemm_simt_kernel<false, false, SPLIT>, grid, GT, 0, 1, st, g, part);
}

// The shares of K, by the time of the busiest SM (us). Measured: 16 of K of one block take 1.33 us, of two
// on an SM 0.89 each, of more 0.82 each (there is no load latency left to hide); a join takes 2.5 and
// 0.0055 for each share of a tile, whose sums go through the L2, the way out of undivided tiles 6. 512 x 1000 x 768: 7 shares 22 us, one
// 68, 16 23; 2048 x 2048 x 512: 2 shares 101 us, one 114, 8 115.
int simt_split(int64_t tiles, int64_t K, int num_sms) {
  int best = 1;
  double least = 0;
  for (int s = 1; s <= kMaxSplit && (s == 1 || (K / s >= 2 * GK && tiles * s <= kMaxShares)); ++s) {
    const int64_t blocks = (tiles * s + num_sms - 1) / num_sms, steps = (K + (int64_t)s * GK - 1) / (s * GK);
    const double t = (double)blocks * steps * (blocks == 1 ? 1.33 : blocks == 2 ? 0.89 : 0.82) + (s > 1 ? 2.5 + 0.0055 * tiles * s : 6);
    if (s == 1 || t < least) {
      least = t;
      best = s;
    }
  }
  return best;
}

// dz = dy * act'(z), and its column sums. 8 columns per thread, `lx` threads side by side (a row's
// 16 lx bytes at a time, for the HBM's sake), 256 / lx rows; the block takes every gridDim.y-th such
// group of rows and adds its rows' sums in order into one row of `part`. VEC: dy's rows hold whole
// 16-byte vectors.
template <typename T, int ACT, bool VEC>
__global__ void __launch_bounds__(256) linear_dz_kernel(const T* dy, int64_t ld_dy, const T* z, int64_t M, int N, T* dz,
                                                        int64_t ld_dz, float* part, int lx) {
  constexpr int U = 4;   // rows in flight
  __shared__ float s[256 * 9];                     // 8 sums a thread, 9 apart
  if (sizeof(T) == 2) pdl_start();   // (before FMA products: see gemm_join_kernel)
  pdl_wait();
  const int ly = 256 / lx, c = threadIdx.x % lx, r = threadIdx.x / lx;
  const int n = (blockIdx.x * lx + c) * 8, cols = min(8, N - n);
  const int64_t step = (int64_t)gridDim.y * ly;
  float sum[8] = {};
  const T* dy_end = dy + (M - 1) * ld_dy + N;
  if (cols > 0) {
    for (int64_t m0 = (int64_t)blockIdx.y * ly + r; m0 < M; m0 += U * step) {
      Vec8<T> a[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t m = m0 + u * step;
        if (m < M) {
          if (VEC) a[u].load_plain(dy + m * ld_dy + n);
          else load8_unaligned(a[u], dy + m * ld_dy + n, dy_end, cols);
          if (ACT != MOE_ACT_NONE) b[u].load_plain(z + m * ld_dz + n);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t m = m0 + u * step;
        if (m >= M) break;
        float v[8], zv[8];
        a[u].to_float(v);
        if constexpr (ACT != MOE_ACT_NONE) {
          b[u].to_float(zv);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= sizeof(T) == 2 ? act_slope_fast<ACT>(zv[i]) : act_slope<ACT>(zv[i]);
        }
        if (dz != nullptr) {   // whole vectors: what lies past N is never read
          Vec8<T> o;
          o.from_float(v);
          o.store(dz + m * ld_dz + n);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += v[i];
      }
    }
  }
  if (part == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) s[threadIdx.x * 9 + i] = sum[i];
  __syncthreads();
  for (int i = threadIdx.x; i < lx * 8; i += 256) {
    const int at = blockIdx.x * lx * 8 + i;
    if (at >= N) break;
    float t = 0.f;
    for (int w = 0; w < ly; ++w) t += s[(w * lx + i / 8) * 9 + i % 8];
    part[(int64_t)blockIdx.y * N + at] = t;
  }
}

// db = the sum of n_part rows: 32 columns per block, 8 threads each, added in order.
template <typename T>
__global__ void __launch_bounds__(256) linear_db_kernel(const float* part, int n_part, int N, T* db) {
  __shared__ float s[8][33];
  const int col = threadIdx.x & 31, r = threadIdx.x >> 5, n = blockIdx.x * 32 + col;
  float t = 0.f;
  if (sizeof(T) == 2) pdl_start();   // (before FMA products: see gemm_join_kernel)
  pdl_wait();
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
  // About 600 blocks (4 on an SM), each with at least 2 rows for a thread. Sums alone in rows of 2 KB
  // (8192 x 7680: 24 us, 31 in rows of 512 bytes and 1200 blocks); with a derivative to compute in
  // rows of 512 (4096 x 2816 SiLU: 12.5 us, 13.9).
  const int lx = act == MOE_ACT_NONE && N > 512 ? 128 : 32, ly = 256 / lx, nx = (N + lx * 8 - 1) / (lx * 8);
  int64_t split = (608 + nx - 1) / nx;
  if (split > (M + 2 * ly - 1) / (2 * ly)) split = (M + 2 * ly - 1) / (2 * ly);
  if (split > kDbSplit) split = kDbSplit;
  const dim3 grid(nx, (unsigned)split);
  const bool vec = N % 8 == 0 && ld_dy % 8 == 0;   // z's and dz's stride is a multiple of 8
  const T *dyp = static_cast<const T*>(dy), *zp = static_cast<const T*>(z);
  T* dzp = static_cast<T*>(dz);
  float* pp = db != nullptr ? part : nullptr;
#define MOE_DZ(A)                                                                                   \
  if (vec) launch_pdl(linear_dz_kernel<T, A, true>, grid, 256, 0, 1, st, dyp, ld_dy, zp, M, N, dzp, ld_dz, pp, lx); \
  else launch_pdl(linear_dz_kernel<T, A, false>, grid, 256, 0, 1, st, dyp, ld_dy, zp, M, N, dzp, ld_dz, pp, lx)
  MOE_ACT_SWITCH(act, MOE_DZ)
#undef MOE_DZ
  if (db != nullptr) launch_pdl(linear_db_kernel<T>, dim3((N + 31) / 32), 256, 0, 1, st, part, (int)split, N, static_cast<T*>(db));
  return cudaGetLastError();
}

}  // namespace

size_t gemm_simt_part_bytes(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = ((M + GM - 1) / GM) * ((N + GN - 1) / GN), most = K / (2 * GK) < kMaxSplit ? K / (2 * GK) : kMaxSplit;
  if (most < 2) return 0;
  return (size_t)(tiles * most < kMaxShares ? tiles * most : kMaxShares) * GM * GN * 4;
}

cudaError_t launch_gemm_simt(const GemmArgs& g, float* part, int num_sms, cudaStream_t st) {
  const int64_t tm = (g.M + GM - 1) / GM, tn = (g.N + GN - 1) / GN;
  const int split = simt_split(tm * tn, g.K, num_sms);
  TraceScope ts(TP_LINEAR, st);
  if (split <= 1) {
    gemm_layouts<false>(g, nullptr, dim3((unsigned)tm, (unsigned)tn), st);
  } else {
    gemm_layouts<true>(g, part, dim3((unsigned)tm, (unsigned)tn, split), st);
    launch_pdl(gemm_join_kernel, dim3((unsigned)tm, (unsigned)tn, GM / JR), 32 * JR, 0, 1, st, g, part, split);
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
