// Layer norm of rows, with the residual's sum in front of it, and its gradients.
//
//   s = x (+ r),  mean = sum s / N,  var = sum (s - mean)^2 / N,  rstd = 1 / sqrt(var + eps)
//   y = (s - mean) rstd w (+ b)
//   u = dy w,  xh = (s - mean) rstd,  dx = rstd (u - mean(u) - xh mean(u xh)) (+ d_sum)
//   dw = sum_m dy xh,  db = sum_m dy
//
// A row stays on the SM between its sums and its way out, so every operand is read once, but for the backward
// of up to kFewRows rows and of the widest ones, where dw and db are another kernel's, which reads x, the residual and dy
// again. The variance is that of the centred values (no difference of large numbers). Many rows that begin on 16 bytes are
// bound by HBM; few rows, and those that begin anywhere, by latency.
//
// Rows of up to 8192 elements (bf16: 16384) are taken by groups of warps, 16 elements (32) to a thread, in a
// persistent block of up to 16 warps; wider ones by a block each. A thread copies its own elements of the
// rows to come into its own places of shared memory (cp.async), several rows ahead, so that the loads of
// a group go on through its barriers, and nobody waits for another thread's copies. The
// columns being a thread's own for all its rows, the weight's gradient is summed in registers.
#include <mutex>

#include "common.cuh"
#include "launch.cuh"
#include "ops.h"
#include "packed.cuh"
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
__host__ __device__ __forceinline__ int part_ld(int N) { return (N + 3) & ~3; }   // between rows of partial sums
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

// ------------------------------------------------------------------ rows of up to kRowsMaxN elements
constexpr int kRowThreads = 512;   // most threads of a block
// Elements of a row that a thread holds: 16, or 32 of wider bf16 rows.
constexpr int kThin = 16, kThick = 32;
constexpr int kRowsMaxN = kRowThreads * kThin, kThickMaxN = kRowThreads * kThick;
constexpr int kMaxStages = 8;
constexpr int kRing = 200 * 1024;   // shared memory of an SM for the copies

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// the first `bytes` of them, zeros behind
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last n of this thread's groups of copies have arrived.
__device__ __forceinline__ void cp_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
  }
}

__device__ __forceinline__ void word_floats(uint32_t w, float& lo, float& hi) {   // two bf16
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}
// 16 bytes of T as pairs, and back (rounded).
__device__ __forceinline__ void unit_pairs(const uint4& v, uint64_t (&f)[2], float) {
  f[0] = pack2(__uint_as_float(v.x), __uint_as_float(v.y));
  f[1] = pack2(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void unit_pairs(const uint4& v, uint64_t (&f)[4], __nv_bfloat16) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float lo, hi;
    word_floats(w[j], lo, hi);
    f[j] = pack2(lo, hi);
  }
}
__device__ __forceinline__ uint4 pairs_unit(const uint64_t (&f)[2], float) {
  float v[4];
  unpack2(f[0], v[0], v[1]);
  unpack2(f[1], v[2], v[3]);
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pairs_unit(const uint64_t (&f)[4], __nv_bfloat16) {
  Vec8<__nv_bfloat16> v;
  float g[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) unpack2(f[j], g[2 * j], g[2 * j + 1]);
  v.from_float(g);
  return v.v;
}
// The 16 bytes that begin `skip` bytes into two pieces (skip a multiple of 2).
__device__ __forceinline__ uint4 window(const uint4& a, const uint4& b, uint32_t skip) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (skip & 8)
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  if (skip & 4)
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  if (skip & 2)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread's weights for a unit of kIn elements of the row, as they are in memory.
template <typename W, int kIn> struct Weights {
  uint4 v[kIn * sizeof(W) / 16];
  __device__ __forceinline__ void load(const W* p, int n) {
    if (n >= kIn) {
#pragma unroll
      for (int q = 0; q < (int)(kIn * sizeof(W) / 16); ++q) v[q] = reinterpret_cast<const uint4*>(p)[q];
    } else {
      W* e = reinterpret_cast<W*>(v);
#pragma unroll
      for (int i = 0; i < kIn; ++i) e[i] = i < n ? p[i] : W(0.f);
    }
  }
  __device__ __forceinline__ void pairs(uint64_t (&f)[kIn / 2]) const {
    if constexpr (sizeof(W) == 4) {
      const float* e = reinterpret_cast<const float*>(v);
#pragma unroll
      for (int j = 0; j < kIn / 2; ++j) f[j] = pack2(e[2 * j], e[2 * j + 1]);
    } else {
      unit_pairs(v[0], f, W());
    }
  }
};

// A thread's units of a row are 16 bytes each, neighbouring threads' side by side, in the row as in shared
// memory. UNALIGNED (some row does not start on a 16-byte boundary): a unit's copy is the two aligned pieces
// around it, and a row may end inside one. ALIGNED: a thread has each unit as a whole or not at all (5760 wide: 45 us
// forward and 55 backward, 47 and 58 with tests for a row's end inside a unit). FULL: it has all of them (widths of 32 E
// times the warps), which saves every test (8192 x 7680, two blocks on an SM: 95 us forward with them, 91 without).
enum RowMode { UNALIGNED = 0, ALIGNED = 1, FULL = 2 };
template <typename T, int MODE, int E> struct Unit {
  static constexpr int kIn = 16 / sizeof(T), kPairs = kIn / 2, kUnits = E / kIn;   // elements; pairs; of a thread
  static constexpr int kPieces = MODE == UNALIGNED ? 2 : 1;
  // p: the unit's first element; n: elements of the row from there on; end: the tensor's
  static __device__ __forceinline__ void copy(uint32_t at, const T* p, int n, const T* end) {
    if (MODE != UNALIGNED) {
      cp_async16(at, p);
    } else {
      const uintptr_t from = reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15);
      const int64_t there = (int64_t)(reinterpret_cast<uintptr_t>(end) - from);   // up to the tensor's end
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int64_t left = there - 16 * q;
        const int bytes = left >= 16 ? 16 : left > 0 ? (int)left : 0;
        cp_async16(at + q * blockDim.x * 16, reinterpret_cast<const void*>(bytes > 0 ? from + 16 * q : from), bytes);
      }
    }
  }
  // As pairs; elements that the row has not (n < kIn) are 0.
  static __device__ __forceinline__ void read(uint64_t (&f)[kPairs], const uint4* at, const T* p, int n) {
    if constexpr (MODE == UNALIGNED) {
      unit_pairs(window(at[0], at[blockDim.x], (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15)), f, T());
      if (n < kIn) keep(f, n);
    } else {
      unit_pairs(at[0], f, T());
    }
  }
  // Its way out to p. UNALIGNED: the warp's 32 units go through their first pieces (the lane's is at `at`; its
  // operand has been read) into whole vectors at the row's own 16-byte boundaries, and single elements at both
  // ends; every lane of the warp takes part.
  static __device__ __forceinline__ void write(const uint64_t (&f)[kPairs], uint4* at, T* p, int n) {
    const uint4 v = pairs_unit(f, T());
    if constexpr (MODE == UNALIGNED) {
      const int lane = threadIdx.x & 31;
      at[0] = v;
      __syncwarp();
      const uint4* seg = at - lane;
      T* first = p - lane * kIn;
      const int left = n + lane * kIn, bytes = (left < 32 * kIn ? left : 32 * kIn) * (int)sizeof(T);   // of the warp's segment
      const int skip = (int)((16 - (reinterpret_cast<uintptr_t>(first) & 15)) & 15), at16 = skip + 16 * lane;
      if (at16 + 16 <= bytes) *reinterpret_cast<uint4*>(reinterpret_cast<char*>(first) + at16) = window(seg[lane], seg[skip ? lane + 1 : lane], skip);
      // lanes 0 to 7: elements before the first boundary, 8 to 15: behind the last whole vector
      const int tail = bytes > skip ? skip + ((bytes - skip) & ~15) : skip;   // (a segment may end before the boundary)
      const int e = lane < 8 ? lane : tail / (int)sizeof(T) + lane - 8, stop = lane < 8 ? (skip < bytes ? skip : bytes) : bytes;
      if (lane < 16 && e * (int)sizeof(T) < stop) first[e] = reinterpret_cast<const T*>(seg)[e];
      __syncwarp();
    } else {
      *reinterpret_cast<uint4*>(p) = v;
    }
  }
  static __device__ __forceinline__ void keep(uint64_t (&f)[kPairs], int n) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      float lo, hi;
      unpack2(f[j], lo, hi);
      f[j] = pack2(2 * j < n ? lo : 0.f, 2 * j + 1 < n ? hi : 0.f);
    }
  }
};

// A group of warps that takes a row: sums over its threads.
struct Group {
  int index, warps;   // which of the block's, its warps
  // Sums of one or two values, the same in every thread. `s`: the block's 16 pairs, not in use by the call before.
  template <bool TWO> __device__ __forceinline__ float2 sums(float a, float b, float2* s) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      if (TWO) b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (warps == 1) return make_float2(a, b);
    const int lane = threadIdx.x & 31;
    if (lane == 0) s[threadIdx.x >> 5] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + index), "r"(warps * 32) : "memory");
    float2 t = make_float2(0.f, 0.f);
    if ((lane & 15) < warps) t = s[index * warps + (lane & 15)];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
      if (TWO) t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
    }
    return t;
  }
  // ... of four.
  __device__ __forceinline__ float4 sums(float4 v, float4* s) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = add(v, o);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) s[threadIdx.x >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + index), "r"(warps * 32) : "memory");
    v = make_float4(0.f, 0.f, 0.f, 0.f);
    if ((lane & 15) < warps) v = s[index * warps + (lane & 15)];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = add(v, o);
    return v;
  }
  static __device__ __forceinline__ float4 add(const float4& v, int o) {
    return make_float4(v.x + __shfl_xor_sync(0xffffffffu, v.x, o), v.y + __shfl_xor_sync(0xffffffffu, v.y, o),
                       v.z + __shfl_xor_sync(0xffffffffu, v.z, o), v.w + __shfl_xor_sync(0xffffffffu, v.w, o));
  }
};

// y (and the sum). Two sums for each row, the second of centred values, each a barrier of the row's group, which takes R
// rows at a time; 94 to 128 registers. 8192 x 7680 bf16 with a residual: 76 us, 6.6 TB/s, HBM; 4096 x 2048 13.2 us, of
// which 3 are its two ends; one row 2.6 us. Rows that begin anywhere: 8190 x 5001 with a residual 111 us, floor 48: issue
// slots 47 % busy, DRAM 23 %, shared memory 31 %, ten warps on an SM that wait for one another and for their own shifts.
template <typename T, typename W, int MODE, int E, bool RES, int R>
__global__ void __launch_bounds__(kRowThreads, 1) norm_fwd_rows(const NormArgs a, int warps, int stages) {
  extern __shared__ uint4 ring[];
  __shared__ float2 s_sums[2][16];
  using P = Unit<T, MODE, E>;
  constexpr int kIn = P::kIn, kUnits = P::kUnits, kPairs = P::kPairs, kOp = kUnits * P::kPieces, kRow = (1 + RES) * kOp;
  pdl_start();
  const int N = a.N, gt = warps * 32, groups = blockDim.x / gt, tg = threadIdx.x % gt;
  const Group group = {(int)threadIdx.x / gt, warps};
  const int64_t step = (int64_t)gridDim.x * groups * R;
  const int c0 = tg * kIn, n0 = N - c0, next_unit = gt * kIn;   // this thread's first column, elements from there on
  const T *x0 = static_cast<const T*>(a.x) + c0, *r0 = RES ? static_cast<const T*>(a.res) + c0 : nullptr;
  const T *x_end = end_of<T>(a.x, a.M, a.ld_x, N), *r_end = RES ? end_of<T>(a.res, a.M, a.ld_res, N) : nullptr;
  pdl_wait();
  int64_t next = ((int64_t)blockIdx.x * groups + group.index) * R;
  const T *xp = x0 + next * a.ld_x, *rp = RES ? r0 + next * a.ld_res : nullptr;   // row `next`
  auto fetch = [&](int stage) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (next + r < a.M) {
        const uint32_t at = smem_u32(ring + (stage * R + r) * kRow * blockDim.x + threadIdx.x);
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
          const int n = n0 - i * next_unit;
          if (MODE == FULL || n > 0) {
            P::copy(at + i * P::kPieces * blockDim.x * 16, xp + r * a.ld_x + i * next_unit, n, x_end);
            if (RES) P::copy(at + (kOp + i * P::kPieces) * blockDim.x * 16, rp + r * a.ld_res + i * next_unit, n, r_end);
          }
        }
      }
    }
    next += step;
    xp += step * a.ld_x;
    if (RES) rp += step * a.ld_res;
    cp_commit();
  };
  constexpr bool ALL = MODE == FULL || E == kThin;   // as in norm_bwd_rows
  if (ALL && MODE == ALIGNED) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      if (n0 - i * next_unit <= 0)
        for (int s = 0; s < stages * R; ++s)
#pragma unroll
          for (int o = 0; o < 1 + RES; ++o) ring[(s * kRow + o * kOp + i) * blockDim.x + threadIdx.x] = make_uint4(0, 0, 0, 0);
  }
  for (int s = 0; s + 1 < stages; ++s) fetch(s);
  constexpr bool HOLD = E * sizeof(W) <= 64;   // the weights in registers; else read for every row
  Weights<W, kIn> w[HOLD ? kUnits : 1], b[HOLD ? kUnits : 1];
  auto weights = [&](int i, int to) {
    const int n = n0 - i * next_unit;
    if (MODE == FULL || n > 0) {
      w[to].load(static_cast<const W*>(a.w) + c0 + i * next_unit, n);
      if (a.b != nullptr) b[to].load(static_cast<const W*>(a.b) + c0 + i * next_unit, n);
    }
  };
  if (HOLD) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) weights(i, i);
  }
  int stage = 0;
  for (int64_t m = ((int64_t)blockIdx.x * groups + group.index) * R; m < a.M; m += step) {
    fetch(stage == 0 ? stages - 1 : stage - 1);   // (the rows before were taken from there)
    cp_wait(stages - 1);
    uint4* at = ring + stage * R * kRow * blockDim.x + threadIdx.x;
    if (++stage == stages) stage = 0;
    uint64_t f[R][kUnits][kPairs];
    uint64_t t[R] = {};
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int n = n0 - i * next_unit;
        uint4* place = at + (r * kRow + i * P::kPieces) * blockDim.x;
        if (ALL || n > 0) {
          P::read(f[r][i], place, x0 + (m + r) * a.ld_x + i * next_unit, n);
          if (RES) {
            uint64_t g[kPairs];
            P::read(g, place + kOp * blockDim.x, r0 + (m + r) * a.ld_res + i * next_unit, n);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) f[r][i][j] = add2(f[r][i][j], g[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < kPairs; ++j) f[r][i][j] = 0;
        }
        if (RES && a.sum != nullptr && (MODE != ALIGNED || n > 0) && (r == 0 || m + r < a.M))
          P::write(f[r][i], place, static_cast<T*>(a.sum) + (m + r) * a.ld_sum + c0 + i * next_unit, n);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) t[r] = add2(t[r], f[r][i][j]);
      }
    float2 all = group.sums<(R > 1)>(sum2(t[0]), sum2(t[R - 1]), s_sums[0]);
    const float mean[2] = {all.x * a.inv_n, all.y * a.inv_n};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      t[r] = 0;
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int n = n0 - i * next_unit;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) f[r][i][j] = add2(f[r][i][j], both(-mean[r]));
        if (MODE == UNALIGNED && n < kIn) P::keep(f[r][i], n);
        if (MODE == ALIGNED && n <= 0) {
#pragma unroll
          for (int j = 0; j < kPairs; ++j) f[r][i][j] = 0;
        }
#pragma unroll
        for (int j = 0; j < kPairs; ++j) t[r] = fma2(f[r][i][j], f[r][i][j], t[r]);
      }
    }
    all = group.sums<(R > 1)>(sum2(t[0]), sum2(t[R - 1]), s_sums[1]);
    const float rstd[2] = {1.f / sqrtf(all.x * a.inv_n + a.eps), R > 1 ? 1.f / sqrtf(all.y * a.inv_n + a.eps) : 0.f};
    if (tg < R && m + tg < a.M && a.stats != nullptr)
      reinterpret_cast<float2*>(a.stats)[m + tg] = make_float2(tg == 0 ? mean[0] : mean[1], tg == 0 ? rstd[0] : rstd[1]);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int n = n0 - i * next_unit;
      uint64_t g[kPairs], h[kPairs] = {};
      if (!HOLD) weights(i, 0);
      w[HOLD ? i : 0].pairs(g);
      if (a.b != nullptr) b[HOLD ? i : 0].pairs(h);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        uint64_t y[kPairs];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) y[j] = fma2(f[r][i][j], mul2(g[j], both(rstd[r])), h[j]);
        if ((MODE != ALIGNED || n > 0) && (r == 0 || m + r < a.M))
          P::write(y, at + (r * kRow + i * P::kPieces) * blockDim.x, static_cast<T*>(a.y) + (m + r) * a.ld_y + c0 + i * next_unit, n);
      }
    }
  }
  cp_wait(0);
}

// dx, and a block's partial sums of dw and db. x, dy, then the residual (RES) and d_sum (DS) are the operands of a
// stage; the next rows' mean and rstd are asked for a step ahead (86 us, 94 without, at 8192 x 7680 with three operands). One
// barrier for R rows. 8192 x 7680 bf16, four operands: 89 us, 7.0 TB/s, HBM; 97 with the sums' join.
// Rows that begin anywhere: 8190 x 5001 152 us, floor 60, by latency as the forward's. A column's sum takes a group's rows one
// after the other in fp32, M / (blocks x groups) roundings in a row at most, and one for each block in the join.
// 126 to 128 registers, all that 512 threads have: 37 of the 64 forms spill, mostly 4 to 16 bytes a thread, those of 32
// elements with every unit up to 160, that of four unaligned fp32 operands (no call of the Python layer) 256.
template <typename T, typename W, int MODE, int E, bool RES, bool DS, int R>
__global__ void __launch_bounds__(kRowThreads, 1) norm_bwd_rows(const NormBwdArgs a, int warps, int stages) {
  extern __shared__ uint4 ring[];
  __shared__ float4 s_sums[2][16];
  using P = Unit<T, MODE, E>;
  constexpr int kIn = P::kIn, kUnits = P::kUnits, kPairs = P::kPairs, kOp = kUnits * P::kPieces, kOps = 2 + RES + DS, kRow = kOps * kOp;
  pdl_start();
  const int N = a.N, gt = warps * 32, groups = blockDim.x / gt, tg = threadIdx.x % gt;
  const Group group = {(int)threadIdx.x / gt, warps};
  const int64_t step = (int64_t)gridDim.x * groups * R;
  const int c0 = tg * kIn, n0 = N - c0, next_unit = gt * kIn;   // this thread's first column, elements from there on
  const void* const operand[4] = {a.x, a.dy, RES ? a.res : a.d_sum, a.d_sum};
  const int64_t ld[4] = {a.ld_x, a.ld_dy, RES ? a.ld_res : a.ld_ds, a.ld_ds};
  pdl_wait();
  int64_t next = ((int64_t)blockIdx.x * groups + group.index) * R;
  const T *base[kOps], *p[kOps], *end[kOps];   // this thread's part of row 0 and of row `next`
#pragma unroll
  for (int o = 0; o < kOps; ++o) {
    base[o] = static_cast<const T*>(operand[o]) + c0;
    p[o] = base[o] + next * ld[o];
    end[o] = end_of<T>(operand[o], a.M, ld[o], N);
  }
  auto fetch = [&](int stage) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (next + r < a.M) {
        const uint32_t at = smem_u32(ring + (stage * R + r) * kRow * blockDim.x + threadIdx.x);
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
          const int n = n0 - i * next_unit;
          if (MODE == FULL || n > 0) {
#pragma unroll
            for (int o = 0; o < kOps; ++o) P::copy(at + (o * kOp + i * P::kPieces) * blockDim.x * 16, p[o] + r * ld[o] + i * next_unit, n, end[o]);
          }
        }
      }
    }
    next += step;
#pragma unroll
    for (int o = 0; o < kOps; ++o) p[o] += step * ld[o];
    cp_commit();
  };
  // Units that this thread does not have are 0 and add nothing, which costs less than to leave them out (8904 x 4600 bf16, four
  // operands: 87 us, 114; 777 x 1001 fp32 9.1, 9.7), but for 32 elements a thread (4096 x 10000: 126 us, 112).
  constexpr bool ALL = MODE == FULL || E == kThin;
  if (ALL && MODE == ALIGNED) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      if (n0 - i * next_unit <= 0)
        for (int s = 0; s < stages * R; ++s)
#pragma unroll
          for (int o = 0; o < kOps; ++o) ring[(s * kRow + o * kOp + i) * blockDim.x + threadIdx.x] = make_uint4(0, 0, 0, 0);
  }
  for (int s = 0; s + 1 < stages; ++s) fetch(s);
  // KEEP: u and xh of one row stay in registers from the sums to dx; else they are formed again from the copies
  constexpr bool KEEP = E == kThin && R == 1, HOLD = E == kThin;
  Weights<W, kIn> w[HOLD ? kUnits : 1] = {};
  uint64_t dw[kUnits][kPairs], db[kUnits][kPairs];
  auto weights = [&](int i, int to) {
    const int n = n0 - i * next_unit;
    if ((MODE == FULL || n > 0) && a.dx != nullptr) w[to].load(static_cast<const W*>(a.w) + c0 + i * next_unit, n);
  };
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (HOLD) weights(i, i);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) dw[i][j] = db[i][j] = 0;
  }
  int stage = 0, buf = 0;
  int64_t m = ((int64_t)blockIdx.x * groups + group.index) * R;
  float2 coming[R];
#pragma unroll
  for (int r = 0; r < R; ++r) coming[r] = m + r < a.M ? reinterpret_cast<const float2*>(a.stats)[m + r] : make_float2(0.f, 0.f);
  for (; m < a.M; m += step) {
    float2 st[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      st[r] = coming[r];
      if (m + step + r < a.M) coming[r] = reinterpret_cast<const float2*>(a.stats)[m + step + r];
    }
    fetch(stage == 0 ? stages - 1 : stage - 1);
    cp_wait(stages - 1);
    uint4* at = ring + stage * R * kRow * blockDim.x + threadIdx.x;
    if (++stage == stages) stage = 0;
    // unit i of row r: xh, and dy (past the row's end 0, and with it all that is added)
    auto unit = [&](int r, int i, uint64_t (&xh)[kPairs], uint64_t (&d)[kPairs]) {
      const int n = n0 - i * next_unit;
      const float mean = MODE == FULL || n > 0 ? st[r].x : 0.f;   // (no product of 0 and infinity)
      const uint4* place = at + (r * kRow + i * P::kPieces) * blockDim.x;
      P::read(xh, place, base[0] + (m + r) * ld[0] + i * next_unit, n);
      P::read(d, place + kOp * blockDim.x, base[1] + (m + r) * ld[1] + i * next_unit, n);
      if (RES) {
        uint64_t g[kPairs];
        P::read(g, place + 2 * kOp * blockDim.x, base[2] + (m + r) * ld[2] + i * next_unit, n);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) xh[j] = add2(xh[j], g[j]);
      }
#pragma unroll
      for (int j = 0; j < kPairs; ++j) xh[j] = mul2(add2(xh[j], both(-mean)), both(st[r].y));
    };
    auto add_columns = [&](int i, const uint64_t (&xh)[kPairs], const uint64_t (&d)[kPairs]) {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        db[i][j] = add2(db[i][j], d[j]);
        dw[i][j] = fma2(d[j], xh[j], dw[i][j]);
      }
    };
    uint64_t u[KEEP ? kUnits : 1][kPairs], xh[KEEP ? kUnits : 1][kPairs];
    uint64_t t[R] = {}, tx[R] = {};
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int k = KEEP ? i : 0;
        if (ALL || n0 - i * next_unit > 0) {
          unit(r, i, xh[k], u[k]);
          if (KEEP) add_columns(i, xh[k], u[k]);
          uint64_t g[kPairs];
          if (!HOLD) weights(i, 0);
          w[HOLD ? i : 0].pairs(g);
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            u[k][j] = mul2(u[k][j], g[j]);
            t[r] = add2(t[r], u[k][j]);
            tx[r] = fma2(u[k][j], xh[k][j], tx[r]);
          }
        }
      }
    if (KEEP && a.dx == nullptr) continue;
    float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.dx != nullptr) {
      if constexpr (R > 1) {
        c = group.sums(make_float4(sum2(t[0]), sum2(tx[0]), sum2(t[R - 1]), sum2(tx[R - 1])), s_sums[buf]);
      } else {
        const float2 one = group.sums<true>(sum2(t[0]), sum2(tx[0]), reinterpret_cast<float2*>(s_sums[buf]));
        c.x = one.x;
        c.y = one.y;
      }
    }
    buf ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r > 0 && m + r >= a.M) break;
      const uint64_t c1 = both(-(r == 0 ? c.x : c.z) * a.inv_n), c2 = both(-(r == 0 ? c.y : c.w) * a.inv_n), rstd = both(st[r].y);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int n = n0 - i * next_unit, k = KEEP ? i : 0;
        uint4* place = at + (r * kRow + i * P::kPieces) * blockDim.x;
        uint64_t g[kPairs] = {};
        if (ALL || n > 0) {
          if (!KEEP) {
            unit(r, i, xh[k], u[k]);
            add_columns(i, xh[k], u[k]);
            if (!HOLD) weights(i, 0);
            w[HOLD ? i : 0].pairs(g);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
              u[k][j] = mul2(u[k][j], g[j]);
              g[j] = 0;
            }
          }
          if (DS) P::read(g, place + (kOps - 1) * kOp * blockDim.x, base[kOps - 1] + (m + r) * ld[kOps - 1] + i * next_unit, n);
#pragma unroll
          for (int j = 0; j < kPairs; ++j) g[j] = fma2(rstd, fma2(xh[k][j], c2, add2(u[k][j], c1)), g[j]);
        }
        if (a.dx != nullptr && (MODE != ALIGNED || n > 0)) P::write(g, place, static_cast<T*>(a.dx) + (m + r) * a.ld_dx + c0 + i * next_unit, n);
      }
    }
  }
  cp_wait(0);
  if (a.dw == nullptr && a.db == nullptr) return;
  // the groups' sums, added in order: [group][dw, db][column], then a block's partial sums
  __syncthreads();
  const int cols = gt * E;
  float* mine = reinterpret_cast<float*>(ring) + group.index * 2 * cols + c0;
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
#pragma unroll
    for (int h = 0; h < kPairs / 2; ++h) {
      *reinterpret_cast<ulonglong2*>(mine + i * next_unit + 4 * h) = make_ulonglong2(dw[i][2 * h], dw[i][2 * h + 1]);
      *reinterpret_cast<ulonglong2*>(mine + cols + i * next_unit + 4 * h) = make_ulonglong2(db[i][2 * h], db[i][2 * h + 1]);
    }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(ring);
#pragma unroll
  for (int k = 0; k < 2; ++k)
    for (int c = threadIdx.x; c < N; c += blockDim.x) {
      float t = 0.f;
      for (int g = 0; g < groups; ++g) t += all[(g * 2 + k) * cols + c];
      a.part[((int64_t)blockIdx.x * 2 + k) * part_ld(N) + c] = t;
    }
}

// Warps of a group and groups of a block for rows of N elements: no more groups than rows for an SM.
struct RowShape {
  int warps, groups;
  RowShape(int N, int64_t M, int num_sms, int each) : warps((N + 32 * each - 1) / (32 * each)), groups(kRowThreads / 32 / warps) {
    const int64_t rows = (M + num_sms - 1) / num_sms;
    if (groups > rows) groups = (int)rows;
  }
  int threads() const { return warps * groups * 32; }
};
// vec: every row starts on a 16-byte boundary; unit: elements of 16 bytes
RowMode row_mode(int N, bool vec, int unit, int each) { return !vec || N % unit != 0 ? UNALIGNED : N % (32 * each) == 0 ? FULL : ALIGNED; }
// 32 elements to a thread: wider rows than 512 threads of 16 hold (4000 x 16384: 124 us forward and 265 backward by a block
// each, 91 and 149 so; 8000 x 5120, where a block holds one group of 16 and three of 32: 61 and 69 by those of 16, 56 and
// 79 by those of 32). fp32 rows would leave no room to copy ahead.
template <typename T> bool thick(int N, bool vec) { return sizeof(T) == 2 && vec && N % 8 == 0 && N > kRowsMaxN && N <= kThickMaxN; }

// ------------------------------------------------------------------ wide rows
// A block for a row, in registers: bf16 rows above 16384 elements, fp32 rows above 8192, unaligned ones above 8192. 2000 x
// 32768 bf16 145 us with a residual (3.6 TB/s, floor 77), 90 without (39); 4000 x 12288 fp32 143 (116) and 107 (58): a
// block's loads stop while it adds.
template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(1024) norm_fwd_wide(const NormArgs a) {
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

// dx alone, the same way. With the columns below, which read x, the residual and dy too: 2000 x 32768 bf16 332 us with a
// residual (eight passes 155, the floor's five 97), 247 without; 4000 x 12288 fp32 264 and 223. 1024 threads have 64 registers
// each: 76 to 308 bytes a thread are spilled.
template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(1024) norm_dx_wide(const NormBwdArgs a) {
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
    a.part[((int64_t)blockIdx.y * 2 + k) * part_ld(N) + at] = t;
  }
}

// dw and db of few rows, from x and dy themselves: a block owns four vectors of columns, 64 threads each take rows
// in turn, added in an order that M alone sets. One partial sum for every row or two would be as much
// to write and read as the operands (backward of 64 x 8192 bf16 by those 10.4 us, 5.4 so; 100 x 256 5.9, 3.7; 180 x
// 7680 12.3, 9.6; with four rows for a thread, 250 x 1024 6.3, 5.5, but 200 x 100 4.7, 6.3).
constexpr int kFewRows = 192;
template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(256) norm_sums_kernel(const NormBwdArgs a) {
  __shared__ float s[2][64][4][9];
  const int lane = threadIdx.x & 3, r = threadIdx.x >> 2, N = a.N, c = (blockIdx.x * 4 + lane) * 8, n = N - c;
  pdl_start();
  pdl_wait();
  float dw[8], db[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = db[j] = 0.f;
  if (n > 0) {
    const T *x = static_cast<const T*>(a.x), *res = static_cast<const T*>(a.res), *dy = static_cast<const T*>(a.dy);
    const T *x_end = end_of<T>(x, a.M, a.ld_x, N), *r_end = end_of<T>(res, a.M, a.ld_res, N), *y_end = end_of<T>(dy, a.M, a.ld_dy, N);
    constexpr int U = kFewRows / 64;   // a thread's rows, all under way at once
    float2 st[U];
    float f[U][8];
    Vec8<T> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t m = r + 64 * u;
      if (m < a.M) {
        st[u] = reinterpret_cast<const float2*>(a.stats)[m];
        load_sum<T, VEC>(f[u], x + m * a.ld_x, res != nullptr ? res + m * a.ld_res : nullptr, c, n, x_end, r_end);
        load_row<T, VEC>(v[u], dy + m * a.ld_dy, c, n, y_end);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r + 64 * u < a.M) {
        float g[8];
        v[u].to_float(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dw[j] = fmaf(g[j], (f[u][j] - st[u].x) * st[u].y, dw[j]);
          db[j] += g[j];
        }
      }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s[0][r][lane][j] = dw[j];
    s[1][r][lane][j] = db[j];
  }
  __syncthreads();
  // 64 sums, four threads each
  const int sum = threadIdx.x >> 2, k = sum >> 5, col = sum & 31, at = blockIdx.x * 32 + col;
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) t += s[k][lane * 16 + i][col >> 3][col & 7];
  t += __shfl_xor_sync(0xffffffffu, t, 1);
  t += __shfl_xor_sync(0xffffffffu, t, 2);
  W* out = static_cast<W*>(k ? a.db : a.dw);
  if (lane == 0 && out != nullptr && at < N) out[at] = from_f32<W>(t);
}

// dw (blockIdx.y 0) and db (1) from their partial sums, added in an order that their number alone sets:
// 32 columns per block, four to a thread, 32 threads each, whose loads are all under way at once (152 blocks' sums of 777 x
// 1001: backward 9.2 us, 11.0 where a loop waited for each). Bound by latency: 5-8 us of a backward with its launch.
template <typename W>
__global__ void __launch_bounds__(256) norm_join_kernel(const float* part, int n_part, int N, W* dw, W* db) {
  __shared__ float4 s[32][8];
  const int v = threadIdx.x & 7, r = threadIdx.x >> 3, n = blockIdx.x * 32 + v * 4, ld = part_ld(N);
  W* out = blockIdx.y == 0 ? dw : db;
  pdl_start();
  pdl_wait();
  if (out == nullptr) return;
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  if (n < N) {
    constexpr int U = 5;   // of a thread that are under way: all, with a block on each of 152 SMs
    for (int i0 = r; i0 < n_part; i0 += 32 * U) {
      float4 p[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + 32 * u;
        p[u] = i < n_part ? *reinterpret_cast<const float4*>(part + ((int64_t)i * 2 + blockIdx.y) * ld + n) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        t.x += p[u].x;
        t.y += p[u].y;
        t.z += p[u].z;
        t.w += p[u].w;
      }
    }
  }
  s[r][v] = t;
  __syncthreads();
  if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < N) {
    const float* col = reinterpret_cast<const float*>(s) + threadIdx.x;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += col[i * 32];
    out[blockIdx.x * 32 + threadIdx.x] = from_f32<W>(sum);
  }
}

int norm_threads(int N) {
  const int t = ((N + 8 * kVecs - 1) / (8 * kVecs) + 31) & ~31;
  return t;
}

// Whether every row of an operand (if it is there) starts on a 16-byte boundary.
template <typename T> bool whole(const void* p, int64_t ld) { return p == nullptr || ld % (16 / (int)sizeof(T)) == 0; }

// Shared memory above the default size has to be allowed, once for each kernel and device.
template <auto Kernel> cudaError_t allow_ring(int bytes) {
  static std::mutex mu;
  static bool allowed[kMaxDevices];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (allowed[dev]) return cudaSuccess;
  const cudaError_t s = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  allowed[dev] = s == cudaSuccess;
  return s;
}

// A persistent launch: one block on an SM (two with half the ring each: 90 us forward at 8192 x 7680, 77 by one).
struct RowLaunch {
  int grid, threads, warps, stages, smem;
  // each: rows that a group takes at a time; stage: bytes of a thread's places of a stage; join: of what it leaves
  // behind the loop
  RowLaunch(int64_t M, const RowShape& s, int each, int stage, int join, int num_sms) : warps(s.warps) {
    int groups = s.groups;
    while (groups > 1 && warps * 32 * groups * stage > kRing) --groups;   // (each takes a stage at least)
    threads = warps * 32 * groups;
    const int64_t blocks = (M + groups * each - 1) / (groups * each);
    grid = (int)(blocks < num_sms ? blocks : num_sms);
    const int64_t rows = (blocks + grid - 1) / grid;   // of a group, `each` at a time
    stages = kRing / (threads * stage);
    if (stages > kMaxStages) stages = kMaxStages;
    if (stages > rows) stages = (int)rows;
    smem = threads * (stages * stage > join ? stages * stage : join);
  }
};

template <typename T, typename W, int MODE, int E, bool RES, int R> cudaError_t fwd_each(const NormArgs& a, int num_sms, cudaStream_t st) {
  using P = Unit<T, MODE, E>;
  static_assert(16 * R * (1 + RES) * P::kUnits * P::kPieces * kRowThreads <= kRing, "a stage at least");
  const RowLaunch l(a.M, RowShape(a.N, a.M, num_sms, E), R, 16 * R * (1 + RES) * P::kUnits * P::kPieces, 0, num_sms);
  const cudaError_t e = allow_ring<norm_fwd_rows<T, W, MODE, E, RES, R>>(kRing);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_fwd_rows<T, W, MODE, E, RES, R>, dim3(l.grid), l.threads, l.smem, 1, st, a, l.warps, l.stages);
}
template <typename T, typename W, int MODE, int E, bool RES> cudaError_t fwd_rows(const NormArgs& a, int num_sms, cudaStream_t st) {
  // Two rows at a time of bf16, each group four times at least: a group's two barriers for them are the same (without a
  // residual 8000 x 5120: 50 us by one, 41 by two; 10000 x 4096 41, 35; 40000 x 1024 35, 30; with one 8000 x 5120 61,
  // 52; 4096 x 2048 14.4, 13.2). With a residual wider rows leave too few stages (5714 x 7168: 54 us by one, 57 by two), and
  // narrow unaligned ones too much to do (52700 x 777: 109, 113).
  if constexpr (sizeof(T) == 2 && E == kThin) {
    const bool two = !RES || (a.N <= 5120 && (MODE != UNALIGNED || a.N > 4096));
    if (two && a.M >= 4 * num_sms * RowShape(a.N, a.M, num_sms, E).groups) return fwd_each<T, W, MODE, E, RES, 2>(a, num_sms, st);
  }
  return fwd_each<T, W, MODE, E, RES, 1>(a, num_sms, st);
}
template <typename T, typename W, int MODE, int E> cudaError_t fwd_mode(const NormArgs& a, int num_sms, cudaStream_t st) {
  return a.res != nullptr ? fwd_rows<T, W, MODE, E, true>(a, num_sms, st) : fwd_rows<T, W, MODE, E, false>(a, num_sms, st);
}

template <typename T, typename W> cudaError_t norm_fwd(const NormArgs& a, int num_sms, cudaStream_t st) {
  const bool vec = a.M == 1 || (whole<T>(a.x, a.ld_x) && whole<T>(a.y, a.ld_y) && whole<T>(a.res, a.ld_res) && whole<T>(a.sum, a.ld_sum));
  if constexpr (sizeof(T) == 2) {
    if (thick<T>(a.N, vec))
      return row_mode(a.N, vec, 8, kThick) == FULL ? fwd_mode<T, W, FULL, kThick>(a, num_sms, st) : fwd_mode<T, W, ALIGNED, kThick>(a, num_sms, st);
  }
  if (a.N <= kRowsMaxN) {
    switch (row_mode(a.N, vec, 16 / (int)sizeof(T), kThin)) {
      case UNALIGNED: return fwd_mode<T, W, UNALIGNED, kThin>(a, num_sms, st);
      case ALIGNED: return fwd_mode<T, W, ALIGNED, kThin>(a, num_sms, st);
      case FULL: return fwd_mode<T, W, FULL, kThin>(a, num_sms, st);
    }
  }
  const dim3 grid((unsigned)a.M);
  return vec ? launch_pdl(norm_fwd_wide<T, W, true>, grid, norm_threads(a.N), 0, 1, st, a)
             : launch_pdl(norm_fwd_wide<T, W, false>, grid, norm_threads(a.N), 0, 1, st, a);
}

template <typename T, typename W, int MODE, int E, bool RES, bool DS, int R>
cudaError_t bwd_each(const NormBwdArgs& a, int num_sms, int* parts, cudaStream_t st) {
  using P = Unit<T, MODE, E>;

  static_assert(16 * R * (2 + RES + DS) * P::kUnits * P::kPieces * kRowThreads <= (MODE == UNALIGNED && sizeof(T) == 4 && RES && DS ? kRing * 4 / 3 : kRing),
                "a stage at least");
  const RowLaunch l(a.M, RowShape(a.N, a.M, num_sms, E), R, 16 * R * (2 + RES + DS) * P::kUnits * P::kPieces, 2 * E * 4, num_sms);
  const cudaError_t e = allow_ring<norm_bwd_rows<T, W, MODE, E, RES, DS, R>>(kRing);
  if (e != cudaSuccess) return e;
  *parts = l.grid;
  return launch_pdl(norm_bwd_rows<T, W, MODE, E, RES, DS, R>, dim3(l.grid), l.threads, l.smem, 1, st, a, l.warps, l.stages);
}

template <typename T, typename W, int MODE, int E, bool RES, bool DS>
cudaError_t bwd_rows(const NormBwdArgs& a, int num_sms, int* parts, cudaStream_t st) {
  // Two rows at a time as the forward, unless they are four operands or unaligned ones, which leave one stage (8000 x 5120
  // bf16: 59.3 us by one row, 53.9 by two; with a residual 72.1, 61.3; 20000 x 2048 46.5, 42.5; 4096 x 7168 42.8, 39.0).
  if constexpr (sizeof(T) == 2 && E == kThin && !(RES && DS) && MODE != UNALIGNED) {
    if (a.M >= 4 * num_sms * RowShape(a.N, a.M, num_sms, E).groups) return bwd_each<T, W, MODE, E, RES, DS, 2>(a, num_sms, parts, st);
  }
  return bwd_each<T, W, MODE, E, RES, DS, 1>(a, num_sms, parts, st);
}

template <typename T, typename W, int MODE, int E> cudaError_t bwd_mode(const NormBwdArgs& a, int num_sms, int* parts, cudaStream_t st) {
  const bool ds = a.d_sum != nullptr && a.dx != nullptr;
  if (a.res != nullptr)
    return ds ? bwd_rows<T, W, MODE, E, true, true>(a, num_sms, parts, st) : bwd_rows<T, W, MODE, E, true, false>(a, num_sms, parts, st);
  return ds ? bwd_rows<T, W, MODE, E, false, true>(a, num_sms, parts, st) : bwd_rows<T, W, MODE, E, false, false>(a, num_sms, parts, st);
}

template <typename T, typename W> cudaError_t norm_bwd(const NormBwdArgs& a, int num_sms, cudaStream_t st) {
  const bool sums = a.dw != nullptr || a.db != nullptr;
  const bool vec = a.M == 1 || (whole<T>(a.x, a.ld_x) && whole<T>(a.dy, a.ld_dy) && whole<T>(a.res, a.ld_res));
  const bool vdx = a.M == 1 || (vec && whole<T>(a.dx, a.ld_dx) && whole<T>(a.d_sum, a.ld_ds));
  int parts = 0;
  cudaError_t e = cudaSuccess;
  if (sums && a.M <= kFewRows) {   // (before dx, which may be the buffer of an operand)
    const dim3 grid((a.N + 31) / 32);
    e = vec ? launch_pdl(norm_sums_kernel<T, W, true>, grid, 256, 0, 1, st, a) : launch_pdl(norm_sums_kernel<T, W, false>, grid, 256, 0, 1, st, a);
    if (e != cudaSuccess || a.dx == nullptr) return e;
    NormBwdArgs d = a;
    d.dw = d.db = nullptr;
    return norm_bwd<T, W>(d, num_sms, st);
  }
  // (a stage of four unaligned fp32 operands, twice what they have, is more than the ring for 13 warps and up)
  const bool four = sizeof(T) == 4 && row_mode(a.N, vdx, 4, kThin) == UNALIGNED && a.res != nullptr && a.d_sum != nullptr && a.dx != nullptr;
  const bool wide = !thick<T>(a.N, vdx) && a.N > (four ? kRowsMaxN * 3 / 4 : kRowsMaxN);
  if (thick<T>(a.N, vdx)) {
    if constexpr (sizeof(T) == 2)
      e = row_mode(a.N, vdx, 8, kThick) == FULL ? bwd_mode<T, W, FULL, kThick>(a, num_sms, &parts, st)
                                             : bwd_mode<T, W, ALIGNED, kThick>(a, num_sms, &parts, st);
  } else if (!wide) {
    switch (row_mode(a.N, vdx, 16 / (int)sizeof(T), kThin)) {
      case UNALIGNED: e = bwd_mode<T, W, UNALIGNED, kThin>(a, num_sms, &parts, st); break;
      case ALIGNED: e = bwd_mode<T, W, ALIGNED, kThin>(a, num_sms, &parts, st); break;
      case FULL: e = bwd_mode<T, W, FULL, kThin>(a, num_sms, &parts, st); break;
    }
  } else if (sums) {   // columns first: dx may be the buffer of an operand
    int64_t share = (a.M + kNormParts - 1) / kNormParts;
    if (share < 8) share = 8;
    parts = (int)((a.M + share - 1) / share);
    const dim3 grid((a.N + 255) / 256, parts);
    e = vec ? launch_pdl(norm_columns_kernel<T, true>, grid, 256, 0, 1, st, a, share)
            : launch_pdl(norm_columns_kernel<T, false>, grid, 256, 0, 1, st, a, share);
  }
  if (e == cudaSuccess && sums)
    e = launch_pdl(norm_join_kernel<W>, dim3((a.N + 31) / 32, 2), 256, 0, 1, st, (const float*)a.part, parts, a.N,
                   static_cast<W*>(a.dw), static_cast<W*>(a.db));
  if (e != cudaSuccess || !wide || a.dx == nullptr) return e;
  const dim3 grid((unsigned)a.M);
  return vdx ? launch_pdl(norm_dx_wide<T, W, true>, grid, norm_threads(a.N), 0, 1, st, a)
             : launch_pdl(norm_dx_wide<T, W, false>, grid, norm_threads(a.N), 0, 1, st, a);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, int dtype, int w_dtype, int num_sms, cudaStream_t st) {
  TraceScope ts(TP_NORM, st);
  if (dtype == MOE_F32) return norm_fwd<float, float>(a, num_sms, st);
  return w_dtype == MOE_F32 ? norm_fwd<__nv_bfloat16, float>(a, num_sms, st) : norm_fwd<__nv_bfloat16, __nv_bfloat16>(a, num_sms, st);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, int w_dtype, int num_sms, cudaStream_t st) {
  TraceScope ts(TP_NORM_BWD, st);
  if (dtype == MOE_F32) return norm_bwd<float, float>(a, num_sms, st);
  return w_dtype == MOE_F32 ? norm_bwd<__nv_bfloat16, float>(a, num_sms, st) : norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, num_sms, st);
}

}  // namespace moe
