// The linear layer's large bf16 products on CTA pairs (sm_103a), C [Mo, No] = A B^T over Ko:
//   forward  y  = act(x W^T + b) + r    A = x  (K-major),  B = W (K-major)
//   dX       dx = dz W                  A = dz (K-major),  B = W (MN-major: W's rows run along Ko)
//   dW       dw = dz^T x                A = dz (MN-major), B = x (MN-major)
//
// The two CTAs of a cluster compute one 256 x TN tile (TN <= 256, chosen by the host for
// the shape) with tcgen05.mma.cta_group::2: each stages its own 128 rows of A and TN / 2 columns of
// B per 64-deep K block (up to 32 KB, six stages) and holds its 128 x TN fp32 half of the tile in
// tensor memory, two tiles deep. Both CTAs' loads complete on the even CTA's full_bar, whose warp 1
// issues the MMAs.
//   warp 0     TMA producer of this CTA's halves
//   warp 1     TMEM owner; in the even CTA it issues the MMAs
//   warps 2..9 epilogue: two warps per TMEM lane quarter, half of the columns each
// Ragged edges need no code in the main loop: the TMA fills what lies outside with zeros.
//
// Where the tiles do not make whole rounds of the pairs, the last ones are divided along K instead
// of leaving pairs idle: each pair takes an equal run of their K blocks. A run's part of a tile that
// ends in another run is left as fp32 partial sums in the workspace; the run that holds the tile's
// last K block adds them in the order of the pairs (so results repeat bit for bit). A pair works on
// its run's last part first, which is what another may wait for; it only waits for pairs of a lower
// index, which were started before it.
//
// z and y are rounded to bf16 from the fp32 sum, each once. Bound by the tensor pipe: 8192 x 7680 x
// 2048 with its gradients, 773 GFLOP, in 489-520 us, 1.49-1.58 PFLOP/s (cuBLAS sustains 1.71 on one
// large product); 4096 x 2816 x 2048 with SiLU and its gradients, 142 GFLOP, in 118-122 us: 32 us a
// product, of which the tensor pipe works 64-73 %, the rest is the first loads and the last tile's
// way out.
//
// Every wait is bounded (1 s): MOE_ERR_DEVICE_TIMEOUT is recorded and the pair winds down.
#include <string.h>

#include <mutex>

#include "act.cuh"
#include "launch.cuh"
#include "ops.h"
#include "tc_common.cuh"
#include "trace.h"

namespace moe {
namespace {

using namespace tc;

constexpr int TM = 256, HM = 128, BK = 64;
constexpr int MAX_TN = 256, MAX_HN = MAX_TN / 2;   // tile columns, and those of B that a CTA stages
constexpr int STAGES = 6, EW = 8;
constexpr int A_BYTES = HM * BK * 2, STAGE_BYTES = A_BYTES + MAX_HN * BK * 2;
constexpr int SLAB = 64 * 128;                    // 64 x 64 elements, 128-byte swizzle
constexpr int PITCH = 80;                         // staging row: 32 bf16 + 16 bytes (no bank conflicts)
constexpr int EPI_BYTES = 32 * PITCH;
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EW * EPI_BYTES + 1024;
constexpr int THREADS = 32 * (2 + EW);
constexpr int PANEL = 8;                          // M tiles walked together per N tile

struct PairGemm {
  CUtensorMap a, b;
  int64_t Mo;
  int No, nkb, tiles_m, tiles_n;
  int tn;                // tile columns: 32 .. 256, a multiple of 32
  uint32_t idesc, stage_tx;   // MMA shape; bytes that both CTAs load per K block
  int sk_tiles;          // the first sk_tiles tiles are divided along K
  int sk_pairs;          // over this many pairs (each gets at least kMinRun K blocks)
  const __nv_bfloat16 *bias, *res;
  __nv_bfloat16 *z, *c;
  int64_t ld_res, ldc, ld_z;
  bool vec, vec_res;     // rows of c, of res, hold whole 16-byte vectors (z's do)
  uint32_t* header;      // error word, epoch, exit count
  uint32_t* flags;       // [CTA][EW]
  float* part;           // [CTA][EW][128 / 4][32 rows][4 columns]
};

// K blocks [k0, k1) of tile t; part: others hold the rest
struct Seg {
  int t, k0, k1;
};

// The segments of a pair: its run of the divided tiles (the last part, which another pair may wait
// for, then the first, which may wait for another, then the whole tiles between, whose MMAs hide
// that wait), then whole tiles.
struct SegCursor {
  int nkb, tiles, np;
  int64_t u0, u1;      // the run's K blocks
  int next_mid, mid;   // its whole tiles left: [next_mid, mid)
  int t;               // next whole tile
  int state;
  Seg s;
  __device__ SegCursor(const PairGemm& g, int pair, int npairs) {
    nkb = g.nkb;
    tiles = g.tiles_m * g.tiles_n;
    np = npairs;
    const int64_t units = (int64_t)g.sk_tiles * nkb;
    u0 = u1 = 0;
    if (pair < g.sk_pairs) {
      u0 = units * pair / g.sk_pairs;
      u1 = units * (pair + 1) / g.sk_pairs;
    }
    next_mid = mid = 0;
    t = g.sk_tiles + pair;
    state = u1 > u0 ? 0 : 2;
  }
  __device__ bool next() {
    if (state == 0) {
      state = 1;
      s.t = (int)((u1 - 1) / nkb);
      const int64_t first = (int64_t)s.t * nkb;
      s.k1 = (int)(u1 - first);
      s.k0 = u0 > first ? (int)(u0 - first) : 0;
      u1 = first + s.k0;
      return true;
    }
    if (state == 1) {
      state = 2;
      if (u1 > u0) {
        s.t = (int)(u0 / nkb);
        s.k0 = (int)(u0 - (int64_t)s.t * nkb);
        s.k1 = nkb;
        mid = (int)(u1 / nkb);
        next_mid = s.t;
        if (s.k0 > 0) {
          ++next_mid;
          return true;
        }
      }
    }
    s.k0 = 0;
    s.k1 = nkb;
    if (next_mid < mid) {
      s.t = next_mid++;
      return true;
    }
    if (t >= tiles) return false;
    s.t = t;
    t += np;
    return true;
  }
};

__device__ __forceinline__ void tile_coord(const PairGemm& g, int t, int& mi, int& ni) {
  const int per = PANEL * g.tiles_n, panel = t / per, r = t - panel * per;
  const int rows = min(PANEL, g.tiles_m - panel * PANEL);
  ni = r / rows;
  mi = panel * PANEL + r - ni * rows;
}

// A TMA load whose bytes complete on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Lane 0 waits for *flag == value; the answer is the same in all lanes.
__device__ __forceinline__ bool flag_wait(const uint32_t* flag, uint32_t value, int lane, volatile int* abort, int* err) {
  bool ok = true;
  if (lane == 0 && ld_acquire(flag) != value) {
    const uint64_t t0 = global_ns();
    while (ld_acquire(flag) != value) {
      if (*abort) { ok = false; break; }
      if (global_ns() - t0 > kWaitLimitNs) {
        record_error(err, MOE_ERR_DEVICE_TIMEOUT);
        *abort = 1;
        ok = false;
        break;
      }
    }
  }
  ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
  __syncwarp();
  return ok;
}

// A warp's 32 rows x 32 columns between global memory and its staging buffer, 64 bytes per row,
// eight rows per instruction; rows that do not hold whole 16-byte vectors are loaded shifted and
// stored element by element, a row per instruction.
struct Chunk {
  int64_t m0;
  int n, rows, cols;
  __device__ __forceinline__ void load(uint4 (&v)[4], const __nv_bfloat16* p, int64_t ld, bool vec, const __nv_bfloat16* end,
                                       int lane) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + (lane >> 2), q = (lane & 3) * 8;
      if (r < rows && q < cols) {
        const __nv_bfloat16* at = p + (m0 + r) * ld + n + q;
        if (vec) {
          v[i] = *reinterpret_cast<const uint4*>(at);
        } else {
          Vec8<__nv_bfloat16> u;
          load8_unaligned(u, at, end, cols - q);
          v[i] = u.v;
        }
      }
    }
  }
  __device__ __forceinline__ void stage(uint8_t* buf, const uint4 (&v)[4], int lane) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(buf + (i * 8 + (lane >> 2)) * PITCH + (lane & 3) * 16) = v[i];
  }
  __device__ __forceinline__ void store(const uint8_t* buf, __nv_bfloat16* p, int64_t ld, bool vec, int lane) const {
    if (vec) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2), q = lane & 3;
        if (r < rows && q * 8 < cols)
          *reinterpret_cast<uint4*>(p + (m0 + r) * ld + n + q * 8) = *reinterpret_cast<const uint4*>(buf + r * PITCH + q * 16);
      }
    } else if (lane < cols) {
#pragma unroll 8
      for (int r = 0; r < rows; ++r) p[(m0 + r) * ld + n + lane] = *reinterpret_cast<const __nv_bfloat16*>(buf + r * PITCH + lane * 2);
    }
  }
};

__device__ __forceinline__ void pack_row(uint8_t* stage, int lane, const float (&v)[32]) {
  uint4* row = reinterpret_cast<uint4*>(stage + lane * PITCH);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    row[q] = make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                        pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
}
// v += 32 bf16 at p (16-byte aligned)
__device__ __forceinline__ void add_row(float (&v)[32], const void* p) {
  const uint4* row = static_cast<const uint4*>(p);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 u = row[q];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      v[8 * q + 2 * i] += t.x;
      v[8 * q + 2 * i + 1] += t.y;
    }
  }
}

__device__ __forceinline__ const __nv_bfloat16* res_end(const PairGemm& g) { return g.res + (g.Mo - 1) * g.ld_res + g.No; }

// bias, z, activation and residual of this lane's 32 columns, and their way out. `res`: the chunk's
// residual, loaded ahead; `next` and `load_next`: the chunk to load into it.
template <int ACT>
__device__ __forceinline__ void finish_chunk(const PairGemm& g, uint8_t* stage, int lane, float (&v)[32], const Chunk& c,
                                             uint4 (&res)[4], const Chunk& next, bool load_next) {
  if (g.bias != nullptr) {
    if (c.cols == 32) {
      add_row(v, g.bias + c.n);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += i < c.cols ? __bfloat162float(g.bias[c.n + i]) : 0.f;
    }
  }
  if (g.z != nullptr) {
    pack_row(stage, lane, v);
    __syncwarp();
    c.store(stage, g.z, g.ld_z, true, lane);
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = act_fast<ACT>(v[i]);
  if (g.res != nullptr) {
    c.stage(stage, res, lane);
    __syncwarp();
    if (load_next) next.load(res, g.res, g.ld_res, g.vec_res, res_end(g), lane);
    add_row(v, stage + lane * PITCH);
    __syncwarp();
  }
  pack_row(stage, lane, v);
  __syncwarp();
  c.store(stage, g.c, g.ldc, g.vec, lane);
  __syncwarp();
}

template <bool A_MN, bool B_MN, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    linear_pair_kernel(const __grid_constant__ PairGemm g) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[STAGES], empty_bar[STAGES], tfull_bar[2], tempty_bar[2], final_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = (int)cluster_id(), npairs = (int)cluster_count();
  int* err = reinterpret_cast<int*>(g.header);
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem_base = smem_u32(smem);

  pdl_start();
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tfull_bar[b]), 1);
      mbar_init(smem_u32(&tempty_bar[b]), 2 * EW);   // the epilogue warps of both CTAs
    }
    mbar_init(smem_u32(&final_bar), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_sh)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync_all();   // the peer's barriers are initialised before any remote arrival
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem_base = tmem_base_sh;
  const uint32_t epoch = *reinterpret_cast<volatile uint32_t*>(g.header + 1) + 1;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    // the whole warp, one lane issuing, as for the MMAs: alone it took 530 cycles per K block
    const bool one = elect_one();
    const uint32_t full0 = peer_addr(smem_u32(&full_bar[0]), 0);   // the even CTA's
    const int hn = g.tn / 2;
    int stage = 0, loaded = 0;
    uint32_t phase = 0;
    bool ok = true;
    SegCursor cur(g, pair, npairs);
    while (ok && cur.next()) {
      int mi, ni;
      tile_coord(g, cur.s.t, mi, ni);
      const int m0 = mi * TM + HM * (int)rank, n0 = ni * g.tn + hn * (int)rank;
      for (int kb = cur.s.k0; kb < cur.s.k1; ++kb) {
        ok = warp_bar_wait(smem_u32(&empty_bar[stage]), phase ^ 1u, &abort_flag, err);
        if (!ok) break;
        if (one) {
          const uint32_t a_s = smem_base + stage * STAGE_BYTES, b_s = a_s + A_BYTES, bar = full0 + stage * 8;
          if (leader) mbar_arrive_expect_tx(smem_u32(&full_bar[stage]), g.stage_tx);
          const int k0 = kb * BK;
          if (A_MN) {
            tma2d_pair(a_s, &g.a, bar, m0, k0);
            tma2d_pair(a_s + SLAB, &g.a, bar, m0 + 64, k0);
          } else {
            tma2d_pair(a_s, &g.a, bar, k0, m0);
          }
          if (B_MN) {
            tma2d_pair(b_s, &g.b, bar, n0, k0);
            if (hn > 64) tma2d_pair(b_s + SLAB, &g.b, bar, n0 + 64, k0);
          } else {
            tma2d_pair(b_s, &g.b, bar, k0, n0);
          }
        }
        ++loaded;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    // drain: no TMA load may still be writing shared memory when the pair exits
    if (leader && one)
      for (int i = 0; i < STAGES && i < loaded; ++i) {
        if (stage == 0) { stage = STAGES; phase ^= 1u; }
        --stage;
        mbar_wait_bounded(smem_u32(&full_bar[stage]), phase, nullptr, err, kWaitLimitNs);
      }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (leader) {
      const uint32_t idesc = g.idesc;
      constexpr uint32_t hi = sdesc_hi(1024), a_step = A_MN ? 2048 / 16 : 32 / 16, b_step = B_MN ? 2048 / 16 : 32 / 16;
      const uint32_t a0 = sdesc_lo(smem_base, A_MN ? SLAB : 16), b0 = sdesc_lo(smem_base + A_BYTES, B_MN ? SLAB : 16);
      const bool one = elect_one();
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      SegCursor cur(g, pair, npairs);
      for (; ok && cur.next(); ++it) {
        const int b = it & 1;
        ok = warp_bar_wait(smem_u32(&tempty_bar[b]), ((it >> 1) & 1) ^ 1, &abort_flag, err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(b * MAX_TN);
        const int blocks = cur.s.k1 - cur.s.k0;
        for (int kb = 0; kb < blocks; ++kb) {
          ok = warp_bar_wait(smem_u32(&full_bar[stage]), phase, &abort_flag, err);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a_lo = a0 + stage * (STAGE_BYTES / 16), b_lo = b0 + stage * (STAGE_BYTES / 16);
          if (one) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              umma_lo<2>(d_tmem, a_lo + kk * a_step, hi, b_lo + kk * b_step, hi, idesc, (kb | kk) != 0 ? 1u : 0u);
            umma_commit_mc(smem_u32(&empty_bar[stage]), 0x3);
          }
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (one) umma_commit_mc(smem_u32(&tfull_bar[b]), 0x3);
      }
      if (one) {   // every MMA retired before the tensor memory is released
        umma_commit_mc(smem_u32(&final_bar), 0x1);
        mbar_wait_bounded(smem_u32(&final_bar), 0, nullptr, err, kWaitLimitNs);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int ew = warp - 2, lg = warp & 3, hn = g.tn / 2, col0 = (ew >> 2) * hn;
    uint8_t* stage = smem + STAGES * STAGE_BYTES + ew * EPI_BYTES;
    const int slot = (int)blockIdx.x * EW + ew;
    int it = 0;
    SegCursor cur(g, pair, npairs);
    for (; cur.next(); ++it) {
      const int b = it & 1;
      int mi, ni;
      tile_coord(g, cur.s.t, mi, ni);
      const int64_t m0 = (int64_t)mi * TM + HM * (int)rank + lg * 32;
      const int rows = (int)min((int64_t)32, g.Mo - m0), n0 = ni * g.tn + col0;
      const bool live = rows > 0 && n0 < g.No;    // the same for every part of the tile
      const bool owner = cur.s.k1 == g.nkb;
      auto chunk = [&](int c) { return Chunk{m0, n0 + c, rows, min(32, min(hn - c, g.No - n0 - c))}; };
      uint4 res[4];
      if (live && owner && g.res != nullptr) chunk(0).load(res, g.res, g.ld_res, g.vec_res, res_end(g), lane);
      const bool got = mbar_wait_bounded(smem_u32(&tfull_bar[b]), (it >> 1) & 1, &abort_flag, err, kWaitLimitNs);
      if (!__all_sync(0xffffffffu, got)) break;   // warp-uniform: tcgen05.ld is .sync.aligned
      tc_fence_after();
      const uint32_t acc = tmem_base + ((uint32_t)(lg * 32) << 16) + (uint32_t)(b * MAX_TN + col0);
      bool ok = true;
      if (live && !owner) {
        // the tile ends in a later pair's run: leave the partial sums to it
        float4* out = reinterpret_cast<float4*>(g.part) + (int64_t)slot * 32 * 32 + lane;
#pragma unroll 1
        for (int c = 0; c < hn; c += 32) {
          uint32_t u[32];
          tmem_ld32(acc + c, u);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            __stcg(out + (c / 4 + i) * 32, make_float4(__uint_as_float(u[4 * i]), __uint_as_float(u[4 * i + 1]),
                                                       __uint_as_float(u[4 * i + 2]), __uint_as_float(u[4 * i + 3])));
        }
        __threadfence();
        __syncwarp();
        if (lane == 0) st_release(g.flags + slot, epoch);
      } else if (live) {
        // the first pair whose run holds a part of the tile, and the wait for all up to this one
        int q0 = pair;
        if (cur.s.k0 > 0) {
          const int64_t units = (int64_t)g.sk_tiles * g.nkb, first = (int64_t)cur.s.t * g.nkb;
          q0 = (int)(first * g.sk_pairs / units);
          while (units * (q0 + 1) / g.sk_pairs <= first) ++q0;
          for (int q = q0; ok && q < pair; ++q)
            ok = flag_wait(g.flags + (q * 2 + (int)rank) * EW + ew, epoch, lane, &abort_flag, err);
        }
        if (ok) {
#pragma unroll 1
          for (int c = 0; c < hn; c += 32) {
            if (n0 + c >= g.No) break;
            uint32_t u[32];
            float v[32];
            tmem_ld32(acc + c, u);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
#pragma unroll 1
            for (int q = q0; q < pair; ++q) {
              const float4* in =
                  reinterpret_cast<const float4*>(g.part) + ((int64_t)((q * 2 + (int)rank) * EW + ew) * 32 + c / 4) * 32 + lane;
              float4 w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = __ldcg(in + i * 32);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                v[4 * i] += w[i].x;
                v[4 * i + 1] += w[i].y;
                v[4 * i + 2] += w[i].z;
                v[4 * i + 3] += w[i].w;
              }
            }
            finish_chunk<ACT>(g, stage, lane, v, chunk(c), res, chunk(c + 32), c + 32 < hn && n0 + c + 32 < g.No);
          }
        }
      }
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(peer_addr(smem_u32(&tempty_bar[b]), 0));
    }
  }
  __syncthreads();
  cluster_sync_all();   // neither CTA releases its tensor memory while the pair still uses it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
  }
  // the last CTA to leave makes this call's flags stale
  if (g.sk_tiles > 0 && threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(g.header + 2, 1u) == gridDim.x - 1) {
      g.header[2] = 0;
      g.header[1] = epoch;
    }
  }
}

// Columns of a tile and the divided tiles, by the time that the slowest pair takes (us). Measured: a
// K block of a 256 x TN tile takes 0.318 / 0.283 / 0.251 / 0.219 / 0.194 / 0.182 / 0.171 us at TN =
// 256 / 224 / 192 / 160 / 128 / 96 / 64 (block_us); a launch kStart; the last tile's way out kOut at
// 256 columns; the division of tiles kJoin at 256 columns (their fp32 parts go through L2) and
// kPart for each part of a tile. Whole rounds of narrower tiles beat divided ones of 256 where some
// width fits the pairs (4096 x 2816 x 2048: 32 us in 160 or 224 columns, 34 in 256, 37 divided);
// 8192 x 2048 x 7680 is divided (141 us, 157 whole); with few tiles and a long K only a division
// uses the pairs.
constexpr double kStart = 4.5, kOut = 3.0, kJoin = 4.0, kPart = 1.5;
inline double block_us(int tn) {
  const double wide = 0.0625 + 0.001 * tn, narrow = 0.17 + 0.0004 * (tn - 64);
  return wide > narrow ? wide : narrow;
}

int plan(PairGemm& g, int pairs) {
  double best = 1e30;
  int used = pairs;
  for (int tn = 256; tn >= 32; tn -= 32) {
    const int64_t tiles = (int64_t)g.tiles_m * ((g.No + tn - 1) / tn);
    const double block = block_us(tn), out = kOut * tn / 256;
    const int64_t rounds = (tiles + pairs - 1) / pairs;
    double cost = kStart + rounds * g.nkb * block + out;
    int sk_tiles = 0, sk_pairs = 0, use = (int)(tiles < pairs ? tiles : pairs);
    const int64_t rem = tiles % pairs;
    if (rem > 0) {
      // with fewer tiles than pairs all are divided; else the incomplete round's and one round more,
      // so that a run is longer than a tile
      const int64_t divided = tiles < pairs ? tiles : rem + pairs;
      int64_t over = divided * g.nkb / kMinRun;
      if (over > pairs) over = pairs;
      const double parts = over > divided ? (double)over / divided : 1.0;
      const double c = kStart + ((tiles - divided) / pairs * g.nkb + (double)divided * g.nkb / over) * block + out + kJoin * tn / 256 +
                       kPart * parts;
      if (over > rem && c < cost) {
        cost = c;
        sk_tiles = (int)divided;
        sk_pairs = (int)over;
        use = tiles < pairs ? (int)over : pairs;
      }
    }
    if (cost < best) {
      best = cost;
      g.tn = tn;
      g.sk_tiles = sk_tiles;
      g.sk_pairs = sk_pairs;
      used = use;
    }
  }
  g.tiles_n = (g.No + g.tn - 1) / g.tn;
  return used;
}

// B's tensor map: K-major in boxes of 64 along K x half a tile, MN-major of 64 columns x 64 of K.
bool map_b(PairGemm& g, const GemmArgs& a) {
  return a.bk == 1 ? map2d_ld(&g.b, a.b, a.K, a.N, a.bn, BK, g.tn / 2) : map2d_ld(&g.b, a.b, a.N, a.K, a.bk, 64, BK);
}

template <bool A_MN, bool B_MN, int ACT>
int launch_pair(PairGemm& g, const GemmArgs& a, int num_sms, cudaStream_t st) {
  auto kernel = linear_pair_kernel<A_MN, B_MN, ACT>;
  // per device, once (under a lock): the shared-memory attribute and the pairs resident at once
  static std::mutex mu;
  static int occ_dev[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MOE_ERR_CUDA;
  int pairs;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (occ_dev[dev] == 0) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES) != cudaSuccess)
        return MOE_ERR_CUDA;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)(num_sms & ~1));
      cfg.blockDim = dim3(THREADS);
      cfg.dynamicSmemBytes = SMEM_BYTES;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) return MOE_ERR_CUDA;
      occ_dev[dev] = n < kMaxPairs ? n : kMaxPairs;
    }
    pairs = occ_dev[dev];
  }
  pairs = plan(g, pairs);
  g.idesc = idesc_bf16(TM, g.tn, A_MN, B_MN);
  g.stage_tx = 2 * (A_BYTES + (B_MN ? (g.tn > 128 ? 2 : 1) * SLAB : g.tn / 2 * BK * 2));
  if (!map_b(g, a)) return MOE_ERR_CUDA;
  TraceScope ts(TP_LINEAR, st);
  return launch_pdl(kernel, dim3((unsigned)(2 * pairs)), THREADS, SMEM_BYTES, 1, st, g) == cudaSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // namespace

size_t linear_pair_part_bytes() { return (size_t)2 * kMaxPairs * EW * 128 * 32 * 4; }

int launch_linear_pair(int kind, const GemmArgs& a, uint8_t* ws, size_t part, int num_sms, cudaStream_t st) {
  PairGemm g;
  memset(&g, 0, sizeof(g));
  g.Mo = a.M;
  g.No = a.N;
  g.nkb = (int)((a.K + BK - 1) / BK);
  g.tiles_m = (int)((a.M + TM - 1) / TM);
  g.bias = static_cast<const __nv_bfloat16*>(a.bias);
  g.res = static_cast<const __nv_bfloat16*>(a.res);
  g.z = static_cast<__nv_bfloat16*>(a.z_out);
  g.c = static_cast<__nv_bfloat16*>(a.c);
  g.ld_res = a.ld_res;
  g.ldc = a.ldc;
  g.ld_z = a.ld_z;
  g.vec = a.N % 8 == 0 && a.ldc % 8 == 0;
  g.vec_res = a.N % 8 == 0 && a.ld_res % 8 == 0;
  g.header = reinterpret_cast<uint32_t*>(ws);
  g.flags = g.header + 256;
  g.part = reinterpret_cast<float*>(ws + part);
  // A: K-major in boxes of 64 along K x 128 rows; MN-major of 64 rows x 64 of K
  const bool ok = a.ak == 1 ? map2d_ld(&g.a, a.a, a.K, a.M, a.am, BK, HM) : map2d_ld(&g.a, a.a, a.M, a.K, a.ak, 64, BK);
  if (!ok) return MOE_ERR_CUDA;
  if (kind == LINEAR_DX) return launch_pair<false, true, MOE_ACT_NONE>(g, a, num_sms, st);
  if (kind == LINEAR_DW) return launch_pair<true, true, MOE_ACT_NONE>(g, a, num_sms, st);
#define MOE_P(ACT) return launch_pair<false, false, ACT>(g, a, num_sms, st)
  MOE_ACT_SWITCH(a.act, MOE_P)
#undef MOE_P
  return MOE_OK;
}

}  // namespace moe
