// Products of a weight stream with a few token rows (sm_103a): the pieces that the few-token
// layer (decode_tc.cu) and the linear layer's serving form (linear_stream.cu) share. Runs and their
// joins through the workspace are the layer's; the linear layer joins inside a cluster.
//
// With few tokens a product is a stream of weights out of HBM, and everything here serves that
// stream. The weights are the MMA's A operand, 128 weight rows by 64 of K per stage; the tokens
// are B, NT (16 .. 128) rows; the transposed result, 128 weight rows by NT tokens, accumulates in
// tensor memory, two accumulators deep. One warp issues TMA loads into a ring that fills the
// shared memory (about 190 KB in flight per SM, four times what the HBM's latency needs), one
// issues tcgen05.mma, eight warps take the results out.
//
// The K blocks of all tiles are divided evenly over the CTAs whatever the tile count (a "run" of
// blocks each), so that every SM streams the same number of bytes. A run's part of a tile that
// ends in a later run is left as fp32 partial sums in the workspace; the run that holds the
// tile's last K block adds them in the order of the CTAs (results repeat bit for bit). A CTA works
// on its run's last part first, so that what another CTA waits for is done first, and only waits
// for CTAs of a lower index.
//
// Every wait is bounded (1 s); the warps that take results out leave together (a barrier carries
// the verdict), so that none is left at a barrier.
#pragma once

#include "ops.h"
#include "tc_common.cuh"

namespace moe {
namespace stream {

using namespace tc;

constexpr int BM = 128, BK = 64;
constexpr int A_BYTES = BM * BK * 2;
constexpr int CW = 8, CT = CW * 32;          // warps and threads that take results out
constexpr int THREADS = 64 + CT;
constexpr int PITCH = BM + 4;                // floats between token columns of the staged result
constexpr int MAX_STAGES = 12;

template <int NT> struct Cfg {
  static constexpr int STAGE = A_BYTES + NT * BK * 2;
  static constexpr int ACC_BYTES = NT * PITCH * 4;
  static constexpr int TMEM = 2 * NT;                             // NT is a power of two, 16 at least
  // stages that fit beside the staged result and `extra` bytes of tables
  static constexpr int stages(int extra) {
    const int n = (227 * 1024 - 2048 - ACC_BYTES - extra) / STAGE;
    return n < MAX_STAGES ? n : MAX_STAGES;
  }
  static constexpr int smem(int extra) { return 1024 + stages(extra) * STAGE + ACC_BYTES + extra; }
};

struct Bars {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES], tfull[2], tempty[2], final, list, slab_free, peers_ready, peers_done;
  uint32_t tmem;
  volatile int abort;
};

__device__ __forceinline__ void st_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void add_release(uint32_t* p, uint32_t v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// The slow sides of the waits are calls: the kernels' cold code stays short (an instruction line
// that is not cached costs about 0.4 us while the stream saturates the L2).
static __device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, int* err) {
  return mbar_wait_bounded(bar, parity, abort, err, kWaitLimitNs);
}
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  return mbar_try_wait(smem_u32(bar), parity) || bar_wait_slow(smem_u32(bar), parity, abort, err);
}

__device__ __forceinline__ uint32_t ld_relaxed(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void fence_acquire() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }

// One thread waits until the word holds at least `value`.
static __device__ __noinline__ bool word_wait(const uint32_t* p, uint32_t value, volatile int* abort, int* err) {
  const uint64_t t0 = global_ns();
  while (ld_relaxed(p) < value) {
    if (*abort) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      record_error(err, MOE_ERR_DEVICE_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
  fence_acquire();
  return true;
}

// A warp waits until every lane's flag holds `value`; lanes without one pass nullptr. All flags are
// polled at once: behind a saturated L2 a poll takes about 2 us.
static __device__ __noinline__ bool flags_wait(const uint32_t* p, uint32_t value, volatile int* abort, int* err) {
  const uint64_t t0 = global_ns();
  while (true) {
    bool there = true;
    if (p != nullptr) there = ld_relaxed(p) == value;
    if (__all_sync(0xffffffffu, there)) break;
    if (__any_sync(0xffffffffu, *abort != 0)) return false;
    if (__any_sync(0xffffffffu, global_ns() - t0 > kWaitLimitNs)) {
      record_error(err, MOE_ERR_DEVICE_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
  fence_acquire();
  return true;
}

// Index among the CT threads that take results out (a block's last ones), and their barrier.
__device__ __forceinline__ int ct_tid() { return (int)threadIdx.x - (int)(blockDim.x - CT); }
__device__ __forceinline__ void ct_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// The same, and true in all of them if `bad` is true in any.
__device__ __forceinline__ bool ct_any(bool bad) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(bad ? 1u : 0u)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void umma1_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// K blocks [k0, k1) of tile t
struct Seg {
  int64_t t;
  int k0, k1;
};

// CTA `c` of `n` works on its run of the tiles' K blocks, the last part first. With few blocks
// only as many CTAs as get kMinStreamRun of them take part, so no run among them is empty. Where
// whole tiles leave the busiest CTA at most kWholeTiles blocks more than an even share (a join costs
// about as many), the runs end at tiles (`whole`).
struct Run {
  int64_t units, u0, u;
  int nkb, n;
  Seg s;
  __device__ Run(int64_t tiles, int nkb_, int c, int n_cta, bool whole) {
    nkb = nkb_;
    units = tiles * nkb;
    whole = whole && (tiles + n_cta - 1) / n_cta * nkb - units / n_cta <= kWholeTiles;
    n = (int)min((int64_t)n_cta, max((int64_t)1, whole ? tiles : units / kMinStreamRun));
    const bool in = c >= 0 && c < n;
    u0 = !in ? 0 : whole ? tiles * c / n * nkb : units * c / n;
    u = !in ? 0 : whole ? tiles * (c + 1) / n * nkb : units * (c + 1) / n;
  }
  __device__ bool next() {
    if (u <= u0) return false;
    s.t = (u - 1) / nkb;
    const int64_t first = s.t * nkb;
    s.k1 = (int)(u - first);
    s.k0 = u0 > first ? (int)(u0 - first) : 0;
    u = first + s.k0;
    return true;
  }
  // the CTA whose run holds K block `at` of all (of a divided tile)
  __device__ int holder(int64_t at) const {
    int q = (int)(at * n / units);
    while (units * (q + 1) / n <= at) ++q;
    return q;
  }
};

// Position in the ring of stages.
template <int STAGES> struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++stage == STAGES) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// Set-up by all threads: barriers, tensor memory. Ends with __syncthreads.
template <int NT, int STAGES>
__device__ __forceinline__ void setup(Bars& b, int warp, int cluster = 1) {
  if (threadIdx.x == 0) {
    b.abort = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&b.full[s]), 1);
      mbar_init(smem_u32(&b.empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&b.tfull[i]), 1);
      mbar_init(smem_u32(&b.tempty[i]), CW);
    }
    mbar_init(smem_u32(&b.final), 1);
    mbar_init(smem_u32(&b.list), 1);
    mbar_init(smem_u32(&b.slab_free), 1);
    mbar_init(smem_u32(&b.peers_ready), cluster);
    mbar_init(smem_u32(&b.peers_done), cluster);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&b.tmem)),
                 "r"(Cfg<NT>::TMEM)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
}

template <int NT> __device__ __forceinline__ void teardown(Bars& b, int warp) {
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(b.tmem), "r"(Cfg<NT>::TMEM) : "memory");
  }
}

// Wait for the loads that are still in flight (the producer, before it leaves).
template <int STAGES> __device__ __forceinline__ void drain(Bars& b, const Ring<STAGES>& r, int64_t loaded, int* err) {
  // the last min(loaded, STAGES) loads end just before the ring's position
  Ring<STAGES> q = r;
  const int n = loaded < STAGES ? (int)loaded : STAGES;
  for (int i = 0; i < n; ++i) {
    if (q.stage == 0) {
      q.stage = STAGES;
      q.phase ^= 1u;
    }
    --q.stage;
    bar_wait(&b.full[q.stage], q.phase, nullptr, err);
  }
}

// The MMAs of `blocks` K blocks into accumulator it & 1 (`it` counts the tiles of the launch), by
// the whole warp; `one`: this lane issues.
template <int NT, int STAGES>
__device__ __forceinline__ bool mma_tile(Bars& b, uint32_t smem_base, int blocks, Ring<STAGES>& ring, int it, bool one, int* err) {
  constexpr uint32_t idesc = idesc_bf16(BM, NT, false, false), hi = sdesc_hi(1024);
  const uint32_t a0 = sdesc_lo(smem_base, 16);
  const int buf = it & 1;
  if (!warp_bar_wait(smem_u32(&b.tempty[buf]), ((it >> 1) & 1) ^ 1, &b.abort, err)) return false;
  tc_fence_after();
  const uint32_t d_tmem = b.tmem + (uint32_t)(buf * NT);
  for (int kb = 0; kb < blocks; ++kb) {
    if (!warp_bar_wait(smem_u32(&b.full[ring.stage]), ring.phase, &b.abort, err)) return false;
    tc_fence_after();
    const uint32_t a_lo = a0 + ring.stage * (Cfg<NT>::STAGE / 16);
    if (one) {
#pragma unroll
      for (int kk = 0; kk < BK / 16; ++kk)
        umma_lo<1>(d_tmem, a_lo + kk * 2, hi, a_lo + A_BYTES / 16 + kk * 2, hi, idesc, (kb | kk) != 0 ? 1u : 0u);
      umma1_commit(smem_u32(&b.empty[ring.stage]));
    }
    ring.step();
  }
  if (one) umma1_commit(smem_u32(&b.tfull[buf]));
  return true;
}

// The MMA warp's part of a run.
template <int NT, int STAGES>
__device__ __forceinline__ bool mma_run(Bars& b, uint32_t smem_base, Run run, Ring<STAGES>& ring, int& it, bool one,
                                        int* err) {
  for (; run.next(); ++it)
    if (!mma_tile<NT, STAGES>(b, smem_base, run.s.k1 - run.s.k0, ring, it, one, err)) return false;
  return true;
}

// The part of the CT threads in a run. `flags` and `part` are this run's (one word, NT * 128
// floats per CTA; with `scatter` two of each). f.prepare(t) runs before, f.finish(t, acc) after tile t is
// staged: acc[column * PITCH + weight row].
// scatter: tiles that many CTAs share (an output's, few and with a long K) are joined by all of them,
// each a share of the result (f.out4(t, column, row, sum of 4 rows)): one CTA adding up 37 others'
// parts took 25 us.
template <int NT, class F>
__device__ __forceinline__ bool take_run(Bars& b, Run run, int& it, int cta, uint32_t* flags, uint32_t epoch, float* part,
                                         float* acc, int* err, F& f, bool scatter) {
  constexpr int HALF = NT / 2;
  const int cw = (threadIdx.x >> 5) - 2, lane = threadIdx.x & 31, lg = (threadIdx.x >> 5) & 3;
  const int row = lg * 32 + lane, col0 = (cw >> 2) * HALF;
  int64_t shared_tile[2];   // divided tiles of this CTA (scatter): a run has two at most
  int n_shared = 0;
  const int stride = scatter ? 2 : 1;
  for (; run.next(); ++it) {
    const int buf = it & 1;
    const bool divided = run.s.k0 > 0 || run.s.k1 < run.nkb;
    const bool owner = scatter ? !divided : run.s.k1 == run.nkb;
    const int slot = cta * stride + (scatter && run.s.k0 > 0 ? 1 : 0);
    bool ok = bar_wait(&b.tfull[buf], (it >> 1) & 1, &b.abort, err);
    const int q0 = owner && divided ? run.holder(run.s.t * run.nkb) : cta;
    ok = __all_sync(0xffffffffu, ok);
    if (owner)   // the flags of the tile's other CTAs
      for (int q = q0; ok && q < cta; q += 32) ok = flags_wait(q + lane < cta ? flags + q + lane : nullptr, epoch, &b.abort, err);
    if (owner) f.prepare(run.s.t);
    if (ct_any(!ok)) return false;
    __syncwarp();   // the TMEM loads are for whole warps
    tc_fence_after();
    const uint32_t t_base = b.tmem + ((uint32_t)(lg * 32) << 16) + (uint32_t)(buf * NT);
    uint32_t u[HALF / 8][8];
#pragma unroll
    for (int c = 0; c < HALF / 8; ++c) tmem_ld8(t_base + col0 + 8 * c, u[c]);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < HALF; c += 8) {
      const int col = col0 + c;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[c / 8][i]);
      if (owner) {
#pragma unroll 1
        for (int q = q0; q < cta; q += 4) {   // four CTAs' parts in flight, added in order
          const float* in = part + ((int64_t)q * NT + col) * BM + row;
          float w[4][8];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) w[j][i] = q + j < cta ? __ldcg(in + (j * NT + i) * BM) : 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += w[j][i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[(col + i) * PITCH + row] = v[i];
      } else {
        float* out = part + ((int64_t)slot * NT + col) * BM + row;
#pragma unroll
        for (int i = 0; i < 8; ++i) __stcg(out + i * BM, v[i]);
      }
    }
    // the accumulator is read: the next part may use it
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&b.tempty[buf]));
    if (owner) {
      ct_sync();
      f.finish(run.s.t, acc);
      ct_sync();
    } else {
      __threadfence();
      ct_sync();
      if (threadIdx.x == 64) st_release(flags + slot, epoch);
      if (scatter) {
        if (n_shared == 0) shared_tile[0] = run.s.t;
        else shared_tile[1] = run.s.t;
        ++n_shared;
      }
    }
  }
#pragma unroll 1
  for (int i = 0; i < n_shared; ++i) {
    const int64_t t = i == 0 ? shared_tile[0] : shared_tile[1];
    // CTAs q0 .. q1 hold parts of it, the first in its slot 0, the others in their slot 1
    const int q0 = run.holder(t * run.nkb), q1 = run.holder((t + 1) * run.nkb - 1), n = q1 - q0 + 1;
    bool ok = true;
    for (int q = q0; ok && q <= q1; q += 32)
      ok = flags_wait(q + lane <= q1 ? flags + (q + lane) * 2 + (q + lane > q0 ? 1 : 0) : nullptr, epoch, &b.abort, err);
    if (ct_any(!ok)) return false;
    const int all = f.columns() * (BM / 4), lo = all * (cta - q0) / n, hi = all * (cta - q0 + 1) / n;
#pragma unroll 1
    for (int u = lo + ct_tid(); u < hi; u += CT) {
      const int col = u / (BM / 4), r4 = u % (BM / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int q = q0; q <= q1; q += 8) {   // eight CTAs' parts in flight, added in order
        float4 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j] = q + j <= q1 ? __ldcg(reinterpret_cast<const float4*>(
                                   part + ((int64_t)((q + j) * 2 + (q + j > q0 ? 1 : 0)) * NT + col) * BM + r4))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v = make_float4(v.x + w[j].x, v.y + w[j].y, v.z + w[j].z, v.w + w[j].w);
      }
      f.out4(t, col, r4, v);
    }
  }
  return true;
}

// The last CTA of the launch to leave zeroes the counters and makes the flags stale; true in its
// thread 0.
__device__ __forceinline__ bool leave(uint32_t* header, uint32_t epoch) {
  if (threadIdx.x != 0) return false;
  __threadfence();
  if (atomicAdd(header + 2, 1u) != gridDim.x - 1) return false;
  for (int i = 2; i < 8; ++i) header[i] = 0;
  header[1] = epoch;
  return true;
}

}  // namespace stream
}  // namespace moe
