// The whole MoE layer for a few tokens in one cooperative launch (bf16, sm_103a).
//
// The layer is a stream of weights: those of the selected experts and of the shared ones, each
// read once. Four steps share the SMs, the stream running through all of them (stream.cuh):
//   scores    s = x W_r by the eight result warps on the FMA pipes (fp32), each CTA a slab of d;
//             CTA t then sums token t's slabs in their order, ranks the experts and writes the
//             selection. Meanwhile the producer already streams
//   shared    h_s = silu(x W1_s^T) * (x W3_s^T) of the shared experts, which need no selection;
//   hidden    hw_e = w_te silu(..) * (..) of every selected expert for ALL tokens: a token that did
//             not select e has w = 0 and gets zeros. The MMA has idle columns to spare, and so
//   output    y = sum_e hw_e W2_e^T + sum_s h_s W2_s^T (+ residual) is ONE product whose K runs over
//             all selected and shared experts: the weighted sum over experts happens in the
//             accumulator, in a fixed order, and no per-expert result is ever written.
// A hidden tile is 64 gate rows and the 64 up rows beside them (128 MMA rows); the result warps
// pair them in shared memory. The first stages of W2 are loaded before the grid barrier that the
// hidden rows need; only their token operands wait.
//
// h times its gate is rounded to bf16 once (it is an MMA operand; the training path rounds the
// same product for its dW), y once.
#include <string.h>

#include <mutex>

#include "stream.cuh"
#include "trace.h"

namespace moe {
namespace {

using namespace stream;

constexpr int RT = 128;            // rows of W_r that a CTA takes at a time
// tables behind the staged result: selected experts, and the tokens' selections
constexpr int kSlots = kMaxE * 2;                       // uint16 expert of each slot
constexpr int kIdx = kDecodeMaxT * kMaxK * 2;           // uint16 [T][k]
constexpr int kGate = kDecodeMaxT * kMaxK * 4;          // fp32 [T][k]
constexpr int kExtra = kSlots + kIdx + kGate;

struct DecodeTc {
  CUtensorMap w13, w2, ws13, ws2, x, h, hs;
  DecodeArgs a;
  int n_slab, slab;      // CTAs that take a slab of W_r, rows of each
  int groups;            // row groups of a slab (threads side by side)
  uint32_t* header;      // error, epoch, leave count, scores / tokens / hidden arrivals
  uint32_t* flags;       // [3][CTA]
  float* part;           // [3][CTA][NT][128]
  float* score_part;     // [T][n_slab * groups][E]
  __nv_bfloat16 *hbuf, *hsbuf;   // [slot][NT][f], [S][NT][f_s]
};

struct Tables {
  uint16_t* slots;
  uint16_t* idx;
  float* gate;
};

// ------------------------------------------------------------------ scores and selection
// Partial scores of this CTA's slab. Thread (group, column): groups of threads take every
// groups-th row. xs: [RT][NT] floats of shared memory.
template <int NT>
__device__ __forceinline__ void partial_scores(const DecodeTc& p, int cta, float* xs) {
  const moe_dims& D = p.a.dm;
  const int T = (int)D.T, E = D.E, d = D.d, tid = threadIdx.x - 64;
  const int d0 = cta * p.slab, d1 = min(d, d0 + p.slab);
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.a.x);
  const int cols = min(E, CT), group = tid / cols, rows = p.n_slab * p.groups;
  for (int e0 = 0; e0 < E; e0 += CT) {
    const int e = e0 + tid % cols;
    float s[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) s[t] = 0.f;
    for (int r0 = d0; r0 < d1; r0 += RT) {
      const int n = min(RT, d1 - r0);
      ct_sync();
      for (int i = tid; i < n * T; i += CT) {
        const int t = i / n, r = i - t * n;
        xs[r * NT + t] = __bfloat162float(x[(int64_t)t * d + r0 + r]);
      }
      for (int i = tid; i < n * (NT - T); i += CT) xs[(i / (NT - T)) * NT + T + i % (NT - T)] = 0.f;
      ct_sync();
      if (group < p.groups && e < E) {
#pragma unroll 8
        for (int r = group; r < n; r += p.groups) {
          const float w = __ldg(p.a.w_r + (int64_t)(r0 + r) * E + e);
          const float4* xr = reinterpret_cast<const float4*>(xs + r * NT);
#pragma unroll
          for (int t = 0; t < NT; t += 4) {
            const float4 v = xr[t / 4];
            s[t] = fmaf(v.x, w, s[t]);
            s[t + 1] = fmaf(v.y, w, s[t + 1]);
            s[t + 2] = fmaf(v.z, w, s[t + 2]);
            s[t + 3] = fmaf(v.w, w, s[t + 3]);
          }
        }
      }
    }
    if (group < p.groups && e < E) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (t < T) __stcg(p.score_part + ((int64_t)t * rows + cta * p.groups + group) * E + e, s[t]);
    }
  }
}

// Token t's scores into `scores` (shared memory, [E]); `tmp`: [CT] floats of shared memory.
__device__ __forceinline__ void sum_scores(const DecodeTc& p, int t, float* scores, float* tmp) {
  const int E = p.a.dm.E, tid = threadIdx.x - 64;
  if (p.a.logits_in != nullptr) {
    for (int e = tid; e < E; e += CT) scores[e] = p.a.logits_in[(int64_t)t * E + e];
  } else {
    const int rows = p.n_slab * p.groups;
    const float* in = p.score_part + (int64_t)t * rows * E;
    for (int e0 = 0; e0 < E; e0 += CT) {
      // `ng` threads share a column, each summing every ng-th row in order
      const int cols = min(E - e0, CT), ng = CT / cols, g = tid / cols, e = e0 + tid % cols;
      float s = 0.f;
      if (g < ng) {
#pragma unroll 16
        for (int r = g; r < rows; r += ng) s += __ldcg(in + (int64_t)r * E + e);
      }
      ct_sync();
      tmp[tid] = s;
      ct_sync();
      if (tid < cols) {
        for (int i = 1; i < ng; ++i) s += tmp[i * cols + tid];
        scores[e0 + tid] = s;
      }
    }
  }
  ct_sync();
}

// Order-preserving map of a float to uint32, above 0 for every finite one; NaN is ranked last.
__device__ __forceinline__ uint32_t rank_key(float x) {
  if (!(x == x)) return 1u;
  const uint32_t u = __float_as_uint(x + 0.f);   // -0 ranks as +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The k largest of `scores` (+ bias), descending, ties to the lower index, and their gates
// (softmax over the k): one warp. Element i of a lane is expert lane + 32 i, so a lane's first
// largest is its lowest expert.
__device__ __forceinline__ void select_topk(const DecodeTc& p, int t, const float* scores, uint32_t* keys, int lane) {
  const moe_dims& D = p.a.dm;
  const int E = D.E, k = D.k;
  for (int e = lane; e < E; e += 32) {
    float s = scores[e];
    if (p.a.bias != nullptr) s = s + p.a.bias[e];   // one fp32 rounding, as in the routing kernel
    keys[e] = rank_key(s);
  }
  uint32_t my_key = 0, my_e = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t kb = 0, eb = 0xffffffffu;
    for (int e = lane; e < E; e += 32) {
      const uint32_t key = keys[e];
      if (key > kb) {
        kb = key;
        eb = e;
      }
    }
    const uint32_t km = __reduce_max_sync(0xffffffffu, kb);
    const uint32_t em = __reduce_min_sync(0xffffffffu, kb == km ? eb : 0xffffffffu);
    if ((em & 31u) == (uint32_t)lane) keys[em] = 0u;   // taken
    if (j == lane) {
      my_key = km;
      my_e = em;
    }
    __syncwarp();
  }
  const float v = __uint_as_float((my_key & 0x80000000u) ? (my_key & 0x7fffffffu) : ~my_key);
  const float top = __shfl_sync(0xffffffffu, v, 0);
  float w = lane < k ? expf(v - top) : 0.f, sum = w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  w /= sum;
  if (lane < k) {
    const int64_t q = (int64_t)t * k + lane;
    __stcg(reinterpret_cast<int32_t*>(p.a.ws + p.a.L.idx) + q, (int32_t)my_e);
    __stcg(reinterpret_cast<float*>(p.a.ws + p.a.L.gate) + q, w);
    if (p.a.idx_out != nullptr) p.a.idx_out[q] = (int32_t)my_e;
    if (p.a.gate_out != nullptr) p.a.gate_out[q] = w;
  }
}

// The selected experts in ascending order, and the tokens' selections. Returns their number.
// bits: kMaxE / 32 words, count: one int of shared memory.
__device__ __forceinline__ int build_tables(const DecodeTc& p, const Tables& tb, uint32_t* bits, int* count) {
  const moe_dims& D = p.a.dm;
  const int n = (int)D.T * D.k, tid = threadIdx.x - 64;
  if (tid < kMaxE / 32) bits[tid] = 0u;
  ct_sync();
  for (int i = tid; i < n; i += CT) {
    const int e = __ldcg(reinterpret_cast<const int32_t*>(p.a.ws + p.a.L.idx) + i);
    tb.idx[i] = (uint16_t)e;
    tb.gate[i] = __ldcg(reinterpret_cast<const float*>(p.a.ws + p.a.L.gate) + i);
    atomicOr(bits + (e >> 5), 1u << (e & 31));
  }
  ct_sync();
  if (tid < 32) {   // lane i: word i of the bitmap
    const uint32_t w = bits[tid];
    int c = __popc(w);
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (tid >= o) inc += v;
    }
    int at = inc - c;
    for (uint32_t m = w; m != 0u; m &= m - 1u) tb.slots[at++] = (uint16_t)(tid * 32 + __ffs((int)m) - 1);
    if (tid == 31) *count = inc;
  }
  ct_sync();
  return *count;
}

// ------------------------------------------------------------------ results
// A hidden tile: rows 0..63 gate, 64..127 up. slots == nullptr: shared experts (weight 1).
template <int NT> struct HiddenFinish {
  const DecodeTc& p;
  const Tables& tb;
  const bool shared;
  const int per;                   // tiles of an expert
  float* wt;                       // [NT] weights of the tile's expert
  __device__ void prepare(int64_t tile) {
    const int t = threadIdx.x - 64, k = p.a.dm.k;
    if (t < (int)p.a.dm.T) {
      float w = shared ? 1.f : 0.f;
      if (!shared) {
        const int e = tb.slots[tile / per];
        for (int j = 0; j < k; ++j)
          if (tb.idx[t * k + j] == e) w = tb.gate[t * k + j];
      }
      wt[t] = w;
    }
  }
  __device__ void finish(int64_t tile, int, const float* acc) {
    const int T = (int)p.a.dm.T, f = shared ? p.a.dm.f_s : p.a.dm.f;
    const int64_t slot = tile / per;
    const int j0 = (int)(tile - slot * per) * 64, c = ((threadIdx.x - 64) & 31) * 2;
    __nv_bfloat16* out = (shared ? p.hsbuf : p.hbuf) + slot * NT * f + j0 + c;
    for (int t = (threadIdx.x - 64) >> 5; t < T; t += CW) {
      const float w = wt[t];
      float h[2] = {0.f, 0.f};
      if (w != 0.f) {
        const float2 g = *reinterpret_cast<const float2*>(acc + t * PITCH + c);
        const float2 u = *reinterpret_cast<const float2*>(acc + t * PITCH + 64 + c);
        h[0] = w * (silu_f(g.x) * u.x);
        h[1] = w * (silu_f(g.y) * u.y);
      }
      *reinterpret_cast<uint32_t*>(out + (int64_t)t * f) = pack_bf16x2(h[0], h[1]);
    }
  }
};

struct OutputFinish {
  const DecodeTc& p;
  __device__ void prepare(int64_t) {}
  __device__ void finish(int64_t tile, int, const float* acc) {
    const int T = (int)p.a.dm.T, d = p.a.dm.d, tid = threadIdx.x - 64;
    const int q = (tid & 15) * 8, n = (int)tile * BM + q;
    if (n >= d) return;   // d is a multiple of 64
    for (int t = tid >> 4; t < T; t += 16) {
      float v[8], r[8];
      *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(acc + t * PITCH + q);
      *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(acc + t * PITCH + q + 4);
      Vec8<__nv_bfloat16> b;
      const int64_t at = (int64_t)t * d + n;
      if (p.a.residual != nullptr) {   // may be y's own buffer
        b.v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.a.residual) + at);
        b.to_float(r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
      }
      b.from_float(v);
      b.store(static_cast<__nv_bfloat16*>(p.a.y) + at);
    }
  }
};

// ------------------------------------------------------------------ the kernel
template <int NT>
__global__ void __launch_bounds__(THREADS, 1) decode_kernel(const __grid_constant__ DecodeTc p) {
  constexpr int STAGES = Cfg<NT>::stages(kExtra), STAGE = Cfg<NT>::STAGE;
  static_assert(RT * NT * 4 <= Cfg<NT>::ACC_BYTES, "the slab of x is staged where the result is");
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) Bars b;
  __shared__ uint32_t s_bits[kMaxE / 32];
  __shared__ int s_active;
  __shared__ float s_wt[NT];
  const moe_dims& D = p.a.dm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem_base = smem_u32(smem);
  float* acc = reinterpret_cast<float*>(smem + STAGES * STAGE);
  uint8_t* tables = smem + STAGES * STAGE + Cfg<NT>::ACC_BYTES;
  const Tables tb = {reinterpret_cast<uint16_t*>(tables), reinterpret_cast<uint16_t*>(tables + kSlots),
                     reinterpret_cast<float*>(tables + kSlots + kIdx)};
  int* err = reinterpret_cast<int*>(p.header);
  const int cta = (int)blockIdx.x, n_cta = (int)gridDim.x, T = (int)D.T;
  setup<NT, STAGES>(b, warp);
  const uint32_t epoch = *reinterpret_cast<volatile uint32_t*>(p.header + 1) + 1;
  uint32_t* arrived = p.header + 3;   // scores, tokens, hidden

  const int per_h = D.f / 64, per_s = D.S > 0 ? D.f_s / 64 : 0, nkb_d = D.d / 64;
  const int tiles_out = (D.d + BM - 1) / BM;
  auto shared_run = [&]() { return Run((int64_t)D.S * per_s, nkb_d, cta, n_cta); };
  auto hidden_run = [&](int active) { return Run((int64_t)active * per_h, nkb_d, cta, n_cta); };
  auto output_run = [&](int active) { return Run(tiles_out, active * per_h + D.S * per_s, cta, n_cta); };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      Ring<STAGES> ring;
      int64_t loaded = 0;
      bool ok = true;
      auto acquire = [&]() {
        ok = mbar_wait_bounded(smem_u32(&b.empty[ring.stage]), ring.phase ^ 1u, &b.abort, err, kWaitLimitNs);
        if (ok) mbar_arrive_expect_tx(smem_u32(&b.full[ring.stage]), STAGE);
        return ok;
      };
      // 64 gate and 64 up rows of one expert, and the tokens
      auto hidden = [&](Run run, bool shared) {
        const CUtensorMap* wm = shared ? &p.ws13 : &p.w13;
        const int per = shared ? per_s : per_h, f = shared ? D.f_s : D.f;
        while (ok && run.next()) {
          const int slot = (int)(run.s.t / per), j0 = (int)(run.s.t - (int64_t)slot * per) * 64;
          const int e = shared ? slot : tb.slots[slot];
          for (int kb = run.s.k0; kb < run.s.k1 && acquire(); ++kb) {
            const uint32_t a_s = smem_base + ring.stage * STAGE, bar = smem_u32(&b.full[ring.stage]);
            tma3d(a_s, wm, bar, kb * BK, j0, e);
            tma3d(a_s + A_BYTES / 2, wm, bar, kb * BK, f + j0, e);
            tma2d(a_s + A_BYTES, &p.x, bar, kb * BK, 0);
            ring.step();
            ++loaded;
          }
        }
      };
      if (D.S > 0) hidden(shared_run(), true);
      ok = ok && mbar_wait_bounded(smem_u32(&b.list), 0, &b.abort, err, kWaitLimitNs);
      if (ok) {
        const int active = s_active;
        hidden(hidden_run(active), false);
        // the output's weights at once, its tokens' hidden rows once every CTA has written its own
        const int routed = active * per_h;
        Run run = output_run(active), tokens = run;
        auto weights = [&](int64_t tile, int kb) {
          const uint32_t a_s = smem_base + ring.stage * STAGE, bar = smem_u32(&b.full[ring.stage]);
          if (kb < routed) {
            const int slot = kb / per_h;
            tma3d(a_s, &p.w2, bar, (kb - slot * per_h) * BK, (int)tile * BM, tb.slots[slot]);
          } else {
            const int s = (kb - routed) / per_s;
            tma3d(a_s, &p.ws2, bar, (kb - routed - s * per_s) * BK, (int)tile * BM, s);
          }
        };
        auto rows = [&](const Ring<STAGES>& r, int kb) {
          const uint32_t b_s = smem_base + r.stage * STAGE + A_BYTES, bar = smem_u32(&b.full[r.stage]);
          if (kb < routed) {
            const int slot = kb / per_h;
            tma2d(b_s, &p.h, bar, (kb - slot * per_h) * BK, slot * NT);
          } else {
            const int s = (kb - routed) / per_s;
            tma2d(b_s, &p.hs, bar, (kb - routed - s * per_s) * BK, s * NT);
          }
        };
        Ring<STAGES> behind = ring;   // the first stage whose tokens are still to be loaded
        int ahead = 0;
        bool waited = false;
        auto wait_hidden = [&]() {
          ok = word_wait(arrived + 2, (uint32_t)n_cta, false, &b.abort, err);
          asm volatile("fence.proxy.async;" ::: "memory");   // generic writes of other CTAs, read by TMA
          waited = true;
        };
        auto catch_up = [&]() {
          // the same blocks again, from the run's start, for their tokens
          int left = ahead;
          while (left > 0 && tokens.next())
            for (int kb = tokens.s.k0; kb < tokens.s.k1 && left > 0; ++kb, --left) {
              rows(behind, kb);
              behind.step();
            }
        };
        while (ok && run.next()) {
          for (int kb = run.s.k0; kb < run.s.k1 && ok; ++kb) {
            if (!waited && ahead == STAGES) {   // the ring is full of weights
              wait_hidden();
              if (!ok) break;
              catch_up();
            }
            if (!acquire()) break;
            weights(run.s.t, kb);
            if (waited) rows(ring, kb);
            else ++ahead;
            ring.step();
            ++loaded;
          }
        }
        if (ok && !waited) {
          wait_hidden();
          if (ok) catch_up();
        }
      }
      drain<STAGES>(b, ring, loaded, err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (lane == 0) {
      Ring<STAGES> ring;
      int it = 0;
      bool ok = true;
      if (D.S > 0) ok = mma_run<NT, STAGES>(b, smem_base, shared_run(), ring, it, err);
      ok = ok && mbar_wait_bounded(smem_u32(&b.list), 0, &b.abort, err, kWaitLimitNs);
      if (ok) {
        const int active = s_active;
        ok = mma_run<NT, STAGES>(b, smem_base, hidden_run(active), ring, it, err) &&
             mma_run<NT, STAGES>(b, smem_base, output_run(active), ring, it, err);
      }
      umma1_commit(smem_u32(&b.final));   // every MMA retired before the tensor memory is released
      mbar_wait_bounded(smem_u32(&b.final), 0, nullptr, err, kWaitLimitNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ scores, selection, results
    const int64_t part_run = (int64_t)n_cta * NT * BM;
    int it = 0;
    bool ok = true;
    if (p.a.logits_in == nullptr && cta < p.n_slab) {
      partial_scores<NT>(p, cta, acc);
      __threadfence();
      ct_sync();
      if (threadIdx.x == 64) add_release(arrived, 1u);
    }
    if (cta < T) {
      if (p.a.logits_in == nullptr) {
        if (threadIdx.x == 64) ok = word_wait(arrived, (uint32_t)p.n_slab, false, &b.abort, err);
        ok = !ct_any(!ok);
      }
      for (int t = cta; ok && t < T; t += n_cta) {
        ct_sync();
        sum_scores(p, t, acc, acc + kMaxE);
        if (warp == 2) {
          select_topk(p, t, acc, reinterpret_cast<uint32_t*>(acc), lane);
          __threadfence();
          __syncwarp();
          if (lane == 0) add_release(arrived + 1, 1u);
        }
      }
      ct_sync();
    }
    if (ok && D.S > 0) {
      HiddenFinish<NT> f{p, tb, true, per_s, s_wt};
      ok = take_run<NT>(b, shared_run(), it, cta, p.flags, epoch, p.part, acc, err, f);
    }
    if (ok) {
      if (threadIdx.x == 64) ok = word_wait(arrived + 1, (uint32_t)T, false, &b.abort, err);
      ok = !ct_any(!ok);
    }
    if (ok) {
      const int active = build_tables(p, tb, s_bits, &s_active);
      if (threadIdx.x == 64) mbar_arrive(smem_u32(&b.list));
      HiddenFinish<NT> f{p, tb, false, per_h, s_wt};
      ok = take_run<NT>(b, hidden_run(active), it, cta, p.flags + n_cta, epoch, p.part + part_run, acc, err, f);
      if (ok) {
        __threadfence();
        asm volatile("fence.proxy.async;" ::: "memory");
        ct_sync();
        if (threadIdx.x == 64) add_release(arrived + 2, 1u);
        OutputFinish o{p};
        take_run<NT>(b, output_run(active), it, cta, p.flags + 2 * n_cta, epoch, p.part + 2 * part_run, acc, err, o);
      }
    }
  }
  teardown<NT>(b, warp);
  leave(p.header, epoch);
}

template <int NT>
int launch_nt(DecodeTc& p, int num_sms, cudaStream_t st) {
  constexpr int SMEM = Cfg<NT>::smem(kExtra);
  static std::mutex mu;   // per device, once: the shared-memory attribute
  static bool attr_set[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MOE_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!attr_set[dev]) {
      if (cudaFuncSetAttribute(decode_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess)
        return MOE_ERR_CUDA;
      attr_set[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_sms);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;   // the CTAs wait on one another
  at[0].val.cooperative = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  TraceScope ts(TP_DECODE, st);
  return cudaLaunchKernelEx(&cfg, decode_kernel<NT>, p) == cudaSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // namespace

int decode_token_columns(int64_t T) { return T <= 16 ? 16 : T <= 32 ? 32 : 64; }

int launch_decode_tc(const DecodeArgs& a, int num_sms, cudaStream_t st) {
  const moe_dims& D = a.dm;
  const int nt = decode_token_columns(D.T);
  if (num_sms > kMaxStreamCtas) num_sms = kMaxStreamCtas;
  DecodeTc p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  // slabs of at least 8 rows of W_r
  p.slab = (D.d + num_sms - 1) / num_sms;
  if (p.slab < 8) p.slab = 8;
  p.n_slab = (D.d + p.slab - 1) / p.slab;
  p.groups = D.E < CT ? CT / D.E : 1;
  p.header = reinterpret_cast<uint32_t*>(a.ws);
  p.flags = p.header + 256;
  p.part = reinterpret_cast<float*>(a.ws + a.L.part);
  p.score_part = reinterpret_cast<float*>(a.ws + a.L.score_part);
  p.hbuf = reinterpret_cast<__nv_bfloat16*>(a.ws + a.L.h);
  p.hsbuf = reinterpret_cast<__nv_bfloat16*>(a.ws + a.L.hs);
  const int64_t slots = decode_slots(D);
  bool ok = map3d(&p.w13, a.w13, D.d, 2 * (uint64_t)D.f, D.E, 64, 64) && map3d(&p.w2, a.w2, D.f, D.d, D.E, 64, 128) &&
            map2d(&p.x, a.x, D.d, D.T, 64, nt) && map2d(&p.h, p.hbuf, D.f, slots * nt, 64, nt);
  if (D.S > 0)
    ok = ok && map3d(&p.ws13, a.ws13, D.d, 2 * (uint64_t)D.f_s, D.S, 64, 64) &&
         map3d(&p.ws2, a.ws2, D.f_s, D.d, D.S, 64, 128) && map2d(&p.hs, p.hsbuf, D.f_s, (uint64_t)D.S * nt, 64, nt);
  if (!ok) return MOE_ERR_CUDA;
  if (nt == 16) return launch_nt<16>(p, num_sms, st);
  if (nt == 32) return launch_nt<32>(p, num_sms, st);
  return launch_nt<64>(p, num_sms, st);
}

}  // namespace moe
