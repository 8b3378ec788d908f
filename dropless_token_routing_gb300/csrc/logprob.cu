// Log probabilities of given tokens, with entropy and the most probable alternatives, and the
// gradient of the scores.
//
//   m = max x,  S = sum e^(x - m),  D = sum e^(x - m) (x - m)
//   ln p_j = x_j - m - ln S,  H = ln S - D / S
//   d_x_j = g ([j = token] - p_j) - h p_j (ln p_j + H)      g, h: gradients of ln p_token and H
//
// One pass over a row with the running maximum: a thread takes 16 scores at a time (of few rows 32), and its sums
// move to the new maximum when these hold one. Differences x - m are formed before the exponential,
// so scores of any size (a mask of the type's lowest value among them) keep their meaning: -inf is no
// token, a row of nothing else has no distribution (S = 0).
#include "cluster.cuh"
#include "common.cuh"
#include "launch.cuh"
#include "ops.h"
#include "packed.cuh"
#include "trace.h"

namespace moe {
namespace {

constexpr int LT = 256, LW = LT / 32;   // threads and warps of a block
// A thread takes LU vectors of 8 scores at a time: 2, or 4 of few rows, whose blocks are three to an SM at most and have
// long slices (30 x 131072 bf16: 5.8 us by 2, 4.5 by 4; 8 leave too much to a slice's last, partial step: 32000 scores 2.6, 3.4).
// Blocks of an SM. LU = 2: 4096 x 32000 fp32 with entropy 79 us by 5, 81 by 4, 91 by 6; bf16 52, 55, 48; 8192 x 131072
// bf16 without 300 by 5, 315 by 6; with alternatives, 1024 x 131072, 68 by 4, 86 by 3.
template <typename T, int LU, bool ENT, bool TOP>
constexpr int kBlocks = LU == 4 ? 3 : TOP ? 4 : ENT && sizeof(T) == 2 ? 6 : 5;
constexpr int kMaxCluster = 8;
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
  template <bool ENT> __device__ __forceinline__ void warp_join() {   // the warp's, in every lane
    float max = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) max = fmaxf(max, __shfl_xor_sync(0xffffffffu, max, o));
    to(max);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      S += __shfl_xor_sync(0xffffffffu, S, o);
      if (ENT) D += __shfl_xor_sync(0xffffffffu, D, o);
    }
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

// A row is read in 16-byte vectors wherever it starts: place k of it is the k-th element from the 16-byte
// boundary at or below its first one, which is place `lead` (the tensor's own start is a boundary, so the places
// before it are the row before's). (Vectors shifted into place instead: 2000 x 50001 bf16, forward 56 us,
// 39 so; the gradient 276 us, 66.)
template <typename T> struct Places {
  const T* base;
  int lead, end;   // the row's first place, and the one after its last
  __device__ __forceinline__ Places(const T* row, int V) {
    lead = (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(T);
    base = row - lead;
    end = V + lead;
  }
  // places k .. k + 7 (a multiple of 8); those past the end: not loaded
  __device__ __forceinline__ void load(Vec8<T>& v, int k) const {
    if (k + 8 <= end) {
      v.load_plain(base + k);
    } else {
      T* e = reinterpret_cast<T*>(&v);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = k + i < end ? base[k + i] : T(0.f);
    }
  }
  // as numbers, -inf for those that are not the row's
  __device__ __forceinline__ void scores(float (&f)[8], const Vec8<T>& v, int k) const {
    v.to_float(f);
    if (k < lead || k + 8 > end) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < lead || k + i >= end) f[i] = -kInf;
    }
  }
};

// The highest of a thread's vectors (NaN aside): two bf16 at a time
template <int LU> __device__ __forceinline__ float highest(const Vec8<__nv_bfloat16> (&v)[LU]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(v);
  __nv_bfloat162 m = h[0];
#pragma unroll
  for (int i = 1; i < 4 * LU; ++i) m = __hmax2(m, h[i]);
  return fmaxf(__low2float(m), __high2float(m));
}
template <int LU> __device__ __forceinline__ float highest(const Vec8<float> (&v)[LU]) {
  const float* h = reinterpret_cast<const float*>(v);
  float m = h[0];
#pragma unroll
  for (int i = 1; i < 8 * LU; ++i) m = fmaxf(m, h[i]);
  return m;
}
template <int LU> __device__ __forceinline__ float highest(const float (&f)[LU][8]) {
  float m = f[0][0];
#pragma unroll
  for (int i = 1; i < 8 * LU; ++i) m = fmaxf(m, f[i / 8][i % 8]);
  return m;
}
// Adds a thread's LU vectors, the highest of which is `top`, to its sums; ENT: D too.
template <bool ENT, int LU> __device__ __forceinline__ void add_scores(Sums& s, const float (&f)[LU][8], float top) {
  if (top > s.m) s.to(top);
  const uint64_t nm = both(-s.m), l2e = both(kLog2e);
  uint64_t S[2] = {0, 0}, D[2] = {0, 0};   // two chains of additions
#pragma unroll
  for (int u = 0; u < LU; ++u)
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      uint64_t d = add2(pack2(f[u][i], f[u][i + 1]), nm);
      float a, b;
      if (ENT) {
        unpack2(d, a, b);
        d = pack2(max_nan(a, -200.f), max_nan(b, -200.f));
      }
      unpack2(mul2(d, l2e), a, b);
      const uint64_t e = pack2(exp2_fast(a), exp2_fast(b));
      S[u & 1] = add2(S[u & 1], e);
      if (ENT) D[u & 1] = fma2(e, d, D[u & 1]);
    }
  s.S += sum2(add2(S[0], S[1]));
  if (ENT) s.D += sum2(add2(D[0], D[1]));
}

static_assert(kMaxCluster * kMaxTop == LT && LT / 4 == 64, "");
struct alignas(16) TopShared {
  unsigned long long key[LT];          // candidates, unordered
  unsigned long long sorted[kMaxTop];  // this block's alternatives, descending
  unsigned long long warp[2][LW];
  int equal[2][LW];
  float group[64];                     // maxima of 4 threads each
  int thread[LT];                      // threads that hold a candidate
  float bound;
  int threads, count;
};

// The lowest number above x.
__device__ __forceinline__ float next_above(float x) {
  const int b = __float_as_int(x + 0.f);   // -0 is +0
  return __int_as_float(b < 0 ? b - 1 : b + 1);
}

// Fills t.sorted from place `count` on with scores equal to x, in order.
template <typename T>
__device__ __forceinline__ void take_equal(TopShared& t, const Places<T> row, int j0, int j1, float x, int count, int n) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int j = j0, step = 0; j < j1 && count < n; j += LT * 8, step ^= 1) {
    const int k = j + tid * 8;
    uint32_t equal = 0;
    if (k < j1) {
      Vec8<T> v;
      float f[8];
      row.load(v, k);
      row.scores(f, v, k);
#pragma unroll
      for (int i = 0; i < 8; ++i) equal |= (uint32_t)(f[i] == x) << i;
    }
    int before = __popc(equal);   // the warp's, up to this thread's
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += w;
    }
    if (lane == 31) t.equal[step][warp] = before;
    __syncthreads();
    before += count - __popc(equal);
#pragma unroll
    for (int w = 0; w < LW; ++w) {
      const int o = t.equal[step][w];
      count += o;
      if (w < warp) before += o;
    }
    for (; equal != 0u && before < n; equal &= equal - 1, ++before) t.sorted[before] = key_of(x, k + __ffs(equal) - 1 - row.lead);
  }
}

// The n highest keys, one at a time.
template <typename T> __device__ __forceinline__ void take_one_by_one(TopShared& t, const Places<T> row, int j0, int j1, int n) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned long long best = ~0ull, top = ~0ull;
  for (int k = 0; k < n; ++k) {
    if (best == top) {   // this thread's next key
      best = 0;
      for (int j = j0 + tid * 8; j < j1; j += LT * 8) {
        Vec8<T> v;
        float f[8];
        row.load(v, j);
        row.scores(f, v, j);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const unsigned long long key = key_of(f[i], j + i - row.lead);
          if (f[i] > -kInf && key < top) best = max64(best, key);
        }
      }
    }
    top = best;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max64(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) t.warp[k & 1][warp] = top;
    __syncthreads();
    top = t.warp[k & 1][lane % LW];
#pragma unroll
    for (int o = LW / 2; o > 0; o >>= 1) top = max64(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top == 0) break;
    if (tid == 0) t.sorted[k] = top;
  }
}

// The block's n highest keys among places [j0, j1) of the row, descending, into t.sorted (0: no more).
// `mine`: the highest score that this thread took (vectors threadIdx.x, + LT, ..; -inf: none). The n-th highest of
// 64 groups' maxima is no higher than the n-th highest score, and few scores reach it (24 of 131072
// in random order, n = 20): only the scores of threads that hold one are looked at again, by all of
// the block's threads. Where more than 256 reach it, mostly because they are equal to it (a finite mask that leaves
// fewer than n tokens, a row of one value), those above it are taken, and then of those equal to it the first ones (one
// row of 131072 with such a mask 7.2 us, 48 of them 10.6; by one key at a time 40 and 59). Rows where more than 256 are
// above it (in order) are taken one key at a time.
template <typename T>
__device__ __forceinline__ void block_top(TopShared& t, const Places<T>& row, int j0, int j1, float mine, int n) {
  const int tid = threadIdx.x, lane = tid & 31;
  float g = mine;
  g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 1));
  g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
  if ((lane & 3) == 0) t.group[tid >> 2] = g;
  if (tid == 0) t.threads = t.count = 0;
  if (tid < kMaxTop) t.sorted[tid] = 0;
  __syncthreads();
  if (tid < 64) {
    g = t.group[tid];
    int higher = 0;
#pragma unroll
    for (int i = 0; i < 64; i += 4) {
      const float4 o = *reinterpret_cast<const float4*>(&t.group[i]);
      higher += (o.x > g || (o.x == g && i < tid)) + (o.y > g || (o.y == g && i + 1 < tid)) + (o.z > g || (o.z == g && i + 2 < tid)) +
               (o.w > g || (o.w == g && i + 3 < tid));
    }
    if (higher == n - 1) t.bound = g;
  }
  __syncthreads();
  const float bound = t.bound;
  float least = bound;   // of a candidate
  bool above = false;    // ... is above the bound
  int count;
  while (true) {
    const bool holds = mine >= least && mine > -kInf;
    const uint32_t who = __ballot_sync(0xffffffffu, holds);
    int first = 0;
    if (lane == 0 && who != 0u) first = atomicAdd(&t.threads, __popc(who));
    first = __shfl_sync(0xffffffffu, first, 0);
    if (holds) t.thread[first + __popc(who & ((1u << lane) - 1))] = tid;
    __syncthreads();
    const int steps = (j1 - j0 + LT * 8 - 1) / (LT * 8), items = t.threads * steps;
    for (int k = tid; k < items; k += LT) {
      const int j = j0 + t.thread[k / steps] * 8 + k % steps * (LT * 8);
      if (j < j1) {
        Vec8<T> v;
        float f[8];
        row.load(v, j);
        row.scores(f, v, j);
        uint32_t high = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) high |= (uint32_t)(f[i] >= least && f[i] > -kInf) << i;
        if (high != 0u) {
          int at = atomicAdd(&t.count, __popc(high));
          if (at > LT) break;   // too many
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (high >> i & 1) {
              if (at < LT) t.key[at] = key_of(f[i], j + i - row.lead);
              ++at;
            }
        }
      }
    }
    __syncthreads();
    count = t.count;
    if (count <= LT || above) break;
    above = true;
    least = next_above(bound);
    __syncthreads();
    if (tid == 0) t.threads = t.count = 0;
    __syncthreads();
  }
  if (count > LT) {
    take_one_by_one(t, row, j0, j1, n);
    return;
  }
  if (tid < count) {
    const unsigned long long key = t.key[tid];
    int higher = 0;
#pragma unroll 4
    for (int i = 0; i < count; ++i) higher += t.key[i] > key;
    if (higher < n) t.sorted[higher] = key;
  }
  if (above && bound > -kInf) take_equal(t, row, j0, j1, bound, count, n);
}

// A row is a cluster's (one block for many rows): every block takes a slice, the first one joins their sums. Bound by HBM
// for many rows (8192 x 131072 bf16: 301 us, 7.1 TB/s; 4096 x 32000 fp32 with entropy 79 us, 6.6 TB/s; the exponentials
// alone would take 73 % of that time in bf16), by latency for few (one row of 131072 with 20 alternatives: 5.8 us).
template <typename T, int LU, bool ENT, bool TOP>
__global__ void __launch_bounds__(LT, (kBlocks<T, LU, ENT, TOP>)) logprob_kernel(const LogprobArgs a) {
  constexpr int LC = LU * LT * 8;   // scores that a block takes at a time
  __shared__ Sums s_sums[LW];
  __shared__ float2 s_row;       // the row's maximum and ln S
  __shared__ TopShared s_top[1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ctarank(), ranks = nctarank();
  pdl_start();
  pdl_wait();
  const int64_t m = blockIdx.x / ranks;
  const T* first = static_cast<const T*>(a.x) + m * a.ld;
  const Places<T> row(first, a.V);
  const int slice = (int)(((row.end + ranks - 1) / ranks + 7) & ~7u);
  const int j0 = min((int)rank * slice, row.end), j1 = min(j0 + slice, row.end);
  int token = -1;
  float given = 0.f;
  if (rank == 0 && threadIdx.x == 0 && a.logprob != nullptr) {
    token = a.tokens[m];
    if (token >= a.V) token = -1;
    if (token >= 0) given = to_f32(first[token]);
  }

  Sums s = {kLowest, 0.f, 0.f};
  const int mine = j0 + threadIdx.x * 8, whole = (j1 - j0) / LC;   // steps that no thread ends in
  Vec8<T> v[LU];
  if (whole > 0) {
#pragma unroll
    for (int u = 0; u < LU; ++u) v[u].load_plain(row.base + mine + u * LT * 8);
  }
  for (int k = 0; k < whole; ++k) {
    float f[LU][8];
#pragma unroll
    for (int u = 0; u < LU; ++u) v[u].to_float(f[u]);
    float top = highest(v);
    if (k + 1 < whole) {   // the next step's scores are under way while these are added
#pragma unroll
      for (int u = 0; u < LU; ++u) v[u].load_plain(row.base + mine + (k + 1) * LC + u * LT * 8);
    }
    if (mine < row.lead && k == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < row.lead) f[0][i] = -kInf;
      top = highest(f);
    }
    add_scores<ENT>(s, f, top);
  }
  if (j0 + whole * LC < j1) {
    float f[LU][8];
#pragma unroll
    for (int u = 0; u < LU; ++u) {
      const int j = mine + whole * LC + u * LT * 8;
      if (j < j1) row.load(v[u], j);
    }
#pragma unroll
    for (int u = 0; u < LU; ++u) {
      const int j = mine + whole * LC + u * LT * 8;
      row.scores(f[u], v[u], j < j1 ? j : row.end);
    }
    add_scores<ENT>(s, f, highest(f));
  }
  const float top = s.S == 0.f ? -kInf : s.m;
  s.warp_join<ENT>();
  if (lane == 0) s_sums[warp] = s;
  if constexpr (TOP) block_top(s_top[0], row, j0, j1, top, a.n_top);
  if (ranks > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (rank == 0) {
    if (warp == 0) {   // the sums of up to 64 warps
      Sums o[2];   // (both asked for at once)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = lane + 32 * k;
        o[k] = {kLowest, 0.f, 0.f};
        if (ranks > 1 && r < (int)ranks * LW) {
          const uint32_t at = smem_u32(&s_sums[r % LW]);
          o[k].m = peer_ldf(at, r / LW);
          o[k].S = peer_ldf(at + 4, r / LW);
          if (ENT) o[k].D = peer_ldf(at + 8, r / LW);
        } else if (r < LW) {
          o[k] = s_sums[r];
        }
      }
      s = o[0];
      const float max = fmaxf(o[0].m, o[1].m);
      s.to(max);
      o[1].to(max);
      s.S += o[1].S;
      s.D += o[1].D;
      s.warp_join<ENT>();
      const float log_sum = s.S == 0.f ? -kInf : logf(s.S);   // a row without a distribution: -inf
      if (lane == 0) {
        if (a.logprob != nullptr) a.logprob[m] = token < 0 ? 0.f : s.S == 0.f ? -kInf : (given - s.m) - log_sum;
        const float H = ENT && s.S != 0.f ? log_sum - s.D / s.S : 0.f;
        if (a.stats != nullptr) {
          float2* st = reinterpret_cast<float2*>(a.stats) + (a.keep_entropy ? 2 * m : m);
          st[0] = make_float2(s.m, log_sum);
          if (ENT && a.keep_entropy) st[1].x = H;
        }
        if (ENT) a.entropy[m] = H;
        if (TOP) s_row = make_float2(s.m, log_sum);
      }
    }
    if constexpr (TOP) {
      TopShared& t = s_top[0];
      const int r = threadIdx.x / kMaxTop, i = threadIdx.x % kMaxTop;
      unsigned long long key = 0;
      int at = i;   // the key's place
      if (ranks > 1) {
        if (r < (int)ranks) key = (unsigned long long)peer_ld64(smem_u32(&t.sorted[i]), r);
        t.key[threadIdx.x] = key;   // the blocks' lists in a row
        __syncthreads();
        if (key != 0) {
          // the higher keys of every list (its own among them), in the lists' 32 descending places
          int higher[kMaxCluster] = {};
#pragma unroll
          for (int step = 16; step > 0; step >>= 1)
#pragma unroll
            for (int o = 0; o < kMaxCluster; ++o)
              if (t.key[o * kMaxTop + higher[o] + step - 1] > key) higher[o] += step;
          at = 0;
#pragma unroll
          for (int o = 0; o < kMaxCluster; ++o) at += higher[o] + (t.key[o * kMaxTop + higher[o]] > key);
        }
      } else if (r == 0) {
        key = t.sorted[i];
      }
      const int found = __syncthreads_count(key != 0);   // (and s_row is there)
      if (key != 0 && at < a.n_top) {
        const uint32_t b = (uint32_t)(key >> 32);
        const float x = __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
        a.top_idx[m * a.n_top + at] = (int)index_of(key);
        a.top_logprob[m * a.n_top + at] = (x - s_row.x) - s_row.y;
      }
      // places that no key took
      if ((int)threadIdx.x >= found && (int)threadIdx.x < a.n_top) {
        a.top_idx[m * a.n_top + threadIdx.x] = -1;
        a.top_logprob[m * a.n_top + threadIdx.x] = -kInf;
      }
    }
  }
  if (ranks > 1) {   // the first block has read its peers' sums
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
}

constexpr int GU = 4, GC = GU * LT * 8;   // the same of the gradient

// Rows from the last one back: where the gradient follows the forward pass at once, as a loss's does, L2 still
// holds some of the rows read last (4096 x 32000 fp32: both 236 us from the first row on, 233 so; of 2048 x 32000, 262 MB, 32
// are not read again).
// Bound by HBM: 8192 x 131072 bf16 627 us, 4096 x 32000 fp32 with entropy 156 us, both 6.7-6.9 TB/s; with a tenth of the rows
// padding, which are not read, 599 and 150. Rows of the gradient that begin at another place within 16 bytes than the
// scores' go out by single elements: 4096 x 50001 bf16 126 us, from rows 50048 apart 514.
template <typename T>
__global__ void __launch_bounds__(LT) logprob_bwd_kernel(const LogprobBwdArgs a) {
  pdl_start();
  pdl_wait();
  const int64_t m = a.M - 1 - blockIdx.x;
  const T* first = static_cast<const T*>(a.x) + m * a.ld;
  const Places<T> row(first, a.V);
  T* out = static_cast<T*>(a.dx) + m * a.ld_dx - row.lead;   // of place 0
  const bool vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  const float2* kept = reinterpret_cast<const float2*>(a.stats) + (a.keep_entropy ? 2 * m : m);
  const float2 st = kept[0];
  const bool some = !(st.y == -kInf);     // the row has a distribution
  int token = a.d_logprob != nullptr && some ? a.tokens[m] : -1;
  if (token >= a.V) token = -1;
  const float g = token >= 0 ? a.d_logprob[m] : 0.f;
  token += row.lead;                      // its place (no other place counts when g is 0)
  const float h = a.d_entropy != nullptr && some ? a.d_entropy[m] : 0.f, H = h == 0.f ? 0.f : a.keep_entropy ? kept[1].x : a.entropy[m];
  const bool zero = g == 0.f && h == 0.f;
  for (int j0 = (blockIdx.y * GU * LT + threadIdx.x) * 8; j0 < row.end; j0 += gridDim.y * GC) {
    Vec8<T> v[GU];
    if (!zero) {
#pragma unroll
      for (int u = 0; u < GU; ++u)
        if (j0 + u * LT * 8 < row.end) row.load(v[u], j0 + u * LT * 8);
    }
#pragma unroll
    for (int u = 0; u < GU; ++u) {
      const int j = j0 + u * LT * 8;
      if (j >= row.end) break;
      float f[8];
      if (zero) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.f;
      } else {
        v[u].to_float(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float lp = below(f[i], st.x) - st.y, p = exp2_fast(lp * kLog2e);
          const float d = g * ((j + i == token ? 1.f : 0.f) - p);
          f[i] = h != 0.f ? d - h * (p * (lp + H)) : d;
        }
      }
      if (vec && j >= row.lead && j + 8 <= row.end) {
        v[u].from_float(f);
        v[u].store(out + j);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (j + i >= row.lead && j + i < row.end) out[j + i] = from_f32<T>(f[i]);
      }
    }
  }
}

template <typename T, int LU> cudaError_t logprob_lu(const LogprobArgs& a, dim3 grid, int c, cudaStream_t st) {
  const bool ent = a.entropy != nullptr;
  if (a.n_top > 0)
    return ent ? launch_pdl(logprob_kernel<T, LU, true, true>, grid, LT, 0, c, st, a)
               : launch_pdl(logprob_kernel<T, LU, false, true>, grid, LT, 0, c, st, a);
  return ent ? launch_pdl(logprob_kernel<T, LU, true, false>, grid, LT, 0, c, st, a)
             : launch_pdl(logprob_kernel<T, LU, false, false>, grid, LT, 0, c, st, a);
}

template <typename T> cudaError_t logprob(const LogprobArgs& a, int num_sms, cudaStream_t st) {
  // Few rows: clusters, while all blocks are resident (by their registers 4 on an SM with alternatives, 6 of bf16 without, 5 of
  // fp32) and a slice keeps every thread at two vectors. 200 x 131072 bf16: 18 us by 2, 11 by 4, 14 by 8; with 20
  // alternatives 18, 22, 26; fp32 19, 22, 22.
  const int64_t resident = num_sms * (a.n_top > 0 ? 4 : sizeof(T) == 2 ? 6 : 5);
  int c = 1;
  while (c < kMaxCluster && a.M * c * 2 <= resident && a.V > c * LT * 16) c *= 2;
  const dim3 grid((unsigned)(a.M * c));
  return a.M * c <= 3 * num_sms && a.V >= c * 6144 ? logprob_lu<T, 4>(a, grid, c, st) : logprob_lu<T, 2>(a, grid, c, st);
}

template <typename T> cudaError_t logprob_bwd(const LogprobBwdArgs& a, int num_sms, cudaStream_t st) {
  // a block takes a row, or parts of it while there are fewer than 16 blocks for an SM
  int64_t parts = (16 * num_sms + a.M - 1) / a.M;
  const int64_t most = (a.V + GC - 1) / GC;
  if (parts > most) parts = most;
  return launch_pdl(logprob_bwd_kernel<T>, dim3((unsigned)a.M, (unsigned)parts), LT, 0, 1, st, a);
}

}  // namespace

cudaError_t launch_logprob(const LogprobArgs& a, int dtype, int num_sms, cudaStream_t st) {
  TraceScope ts(TP_LOGPROB, st);
  return dtype == MOE_F32 ? logprob<float>(a, num_sms, st) : logprob<__nv_bfloat16>(a, num_sms, st);
}

cudaError_t launch_logprob_bwd(const LogprobBwdArgs& a, int dtype, int num_sms, cudaStream_t st) {
  TraceScope ts(TP_LOGPROB_BWD, st);
  return dtype == MOE_F32 ? logprob_bwd<float>(a, num_sms, st) : logprob_bwd<__nv_bfloat16>(a, num_sms, st);
}

}  // namespace moe
