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
// same product for its dW), y once. Scores, gates and all sums are fp32.
//
// Bound by the stream out of HBM, and with few bytes by the chain scores - selection - hidden rows -
// output, whose steps each wait for all CTAs. Measured: T = 32, d = 7168, 77 to 88 experts selected:
// 6.9-7.8 GB in 1.04-1.17 ms, 6.7 TB/s (the copy rate is 6.8); T = 1, d = 7680, 8 experts and a shared
// one: 857 MB in 145-151 us, 5.7-5.9 TB/s; T = 5, d = 2048, 22 to 27 experts and two shared ones: 416-502
// MB in 89-100 us, 4.7-5.1 TB/s; T = 10, d = 448: 1.8 MB in 22 us, all of it the chain.
#include <string.h>

#include <mutex>

#include "act.cuh"
#include "decode_select.cuh"
#include "trace.h"

namespace moe {
namespace {

using namespace decode;

struct DecodeTc {
  CUtensorMap w13, w2, ws13, ws2, x, h, hs;
  DecodeArgs a;
  Select s;
  uint32_t* header;      // error, epoch, leave count, counters (enum)
  uint32_t* flags;       // [kDecodeRuns + 1][CTA]: the output has two parts per CTA
  float* part;           // [kDecodeRuns + 1][CTA][NT][128]
  __nv_bfloat16 *hbuf, *hsbuf;   // [slot][NT][f], [S][NT][f_s]
};

// ------------------------------------------------------------------ the runs
// In the order in which every CTA works on them. (Dividing the output's K into a first part that
// needs no rows of the slower CTAs, to keep the stream going meanwhile, measured no better: the
// joins of a further run cost what it hides.)
enum RunId { SHARED = 0, HIDDEN, OUTPUT };
// An output tile with parts in kScatter or more CTAs is joined by all of them, with 32 columns and
// more: T = 57, d = 448: 39 us, 48 by one CTA. With 16 columns one CTA is done sooner (T = 5, d =
// 2048: 91 us, 93 by all), and with fewer parts there is no difference.
constexpr int kScatter = 4;
static_assert(OUTPUT + 1 == kDecodeRuns, "");

struct Plan {
  int per_h, per_s, k_sh, nkb_d, tiles_out;   // tiles of an expert, K blocks of the shared ones
  int cta, n_cta, T;
  int total;                                  // routed hidden tiles (after the selection)
  __device__ Plan(const moe_dims& D, int cta_, int n_cta_) {
    per_h = D.f / 64;
    per_s = D.S > 0 ? D.f_s / 64 : 1;
    k_sh = D.S * per_s;
    nkb_d = D.d / 64;
    tiles_out = (D.d + BM - 1) / BM;
    cta = cta_;
    n_cta = n_cta_;
    T = (int)D.T;
    total = 0;
  }
  __device__ void select(int active) { total = active * per_h; }
  // The CTAs that select for a token leave the shared experts to the others: behind a stream's
  // loads their own would wait.
  __device__ Run run(int r) const {
    const int tiles = r == SHARED ? k_sh : r == HIDDEN ? total : tiles_out;
    const int nkb = r == OUTPUT ? k_sh + total : nkb_d;
    const int skip = r == SHARED ? T : 0;
    return Run(tiles, nkb, cta - skip, n_cta - skip, r != OUTPUT);
  }
};

// Consecutive K blocks of the output: the shared experts' first, then the selected ones'.
struct Blocks {
  bool shared;
  int slot, at, per;   // block `at` of the `per` of an expert
  __device__ Blocks(const Plan& plan, int kb) {
    shared = kb < plan.k_sh;
    per = shared ? plan.per_s : plan.per_h;
    if (!shared) kb -= plan.k_sh;
    slot = kb / per;
    at = kb - slot * per;
  }
  __device__ void step(const Plan& plan) {
    if (++at < per) return;
    at = 0;
    ++slot;
    if (shared && slot * per == plan.k_sh) {
      shared = false;
      slot = 0;
      per = plan.per_h;
    }
  }
};

// ------------------------------------------------------------------ results
// What becomes of a tile: SHARED, HIDDEN: rows 0..63 gate, 64..127 up -> hidden rows; OUTPUT: y.
template <int NT> struct Finish {
  const DecodeTc& p;
  const Tables& tb;
  const Plan& plan;
  float* wt;                       // [NT] weights of a hidden tile's expert
  int r;
  __device__ void prepare(int64_t tile) {
    const int t = threadIdx.x - 64, k = p.a.dm.k;
    if (r != OUTPUT && t < plan.T) {
      float w = r == SHARED ? 1.f : 0.f;
      if (r != SHARED) {
        const int e = tb.slots[(int)tile / plan.per_h];
#pragma unroll 4
        for (int j = t * k; j < t * k + k; ++j)
          if (tb.idx[j] == e) w = tb.gate[j];
      }
      wt[t] = w;
    }
  }
  __device__ void finish(int64_t tile, const float* acc) {
    const int T = plan.T, tid = threadIdx.x - 64;
    if (r != OUTPUT) {
      const int f = r == SHARED ? p.a.dm.f_s : p.a.dm.f, per = r == SHARED ? plan.per_s : plan.per_h;
      const int at = (int)tile, slot = at / per, c = (tid & 31) * 2;
      __nv_bfloat16* out = (r == SHARED ? p.hsbuf : p.hbuf) + (int64_t)slot * NT * f + (at - slot * per) * 64 + c;
#pragma unroll 4
      for (int t = tid >> 5; t < T; t += CW) {
        const float w = wt[t];
        float h0 = 0.f, h1 = 0.f;
        if (w != 0.f) {
          const float2 g = *reinterpret_cast<const float2*>(acc + t * PITCH + c);
          const float2 u = *reinterpret_cast<const float2*>(acc + t * PITCH + 64 + c);
          h0 = w * (act_fast<MOE_ACT_SILU>(g.x) * u.x);
          h1 = w * (act_fast<MOE_ACT_SILU>(g.y) * u.y);
        }
        *reinterpret_cast<uint32_t*>(out + (int64_t)t * f) = pack_bf16x2(h0, h1);
      }
    } else {
#pragma unroll 1
      for (int t = tid >> 5; t < T; t += CW)
        out4(tile, t, (tid & 31) * 4, *reinterpret_cast<const float4*>(acc + t * PITCH + (tid & 31) * 4));
    }
  }
  __device__ int columns() const { return plan.T; }
  // outputs q .. q + 3 of a tile, token t
  __device__ void out4(int64_t tile, int t, int q, float4 v) {
    const int d = p.a.dm.d, n = (int)tile * BM + q;
    if (n >= d) return;   // d is a multiple of 64
    const int64_t at = (int64_t)t * d + n;
    if (p.a.residual != nullptr) {   // may be y's own buffer
      const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.a.residual) + at);
      const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
      const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
      v = make_float4(v.x + a.x, v.y + a.y, v.z + b.x, v.w + b.y);
    }
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.a.y) + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
};

// ------------------------------------------------------------------ the kernel
template <int NT>
__global__ void __launch_bounds__(THREADS, 1) decode_kernel(const __grid_constant__ DecodeTc p) {
  constexpr int STAGES = Cfg<NT>::stages(kExtra), STAGE = Cfg<NT>::STAGE, SLAB0 = STAGES - 3;
  static_assert(RT * NT * 4 <= Cfg<NT>::ACC_BYTES, "the slab of x is staged where the result is");
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) Bars b;
  __shared__ uint32_t s_bits[kMaxE / 32];
  __shared__ int s_active;
  __shared__ float s_wt[NT];
  __shared__ uint32_t s_top[2 * kMaxK];
  const moe_dims& D = p.a.dm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem_base = smem_u32(smem);
  float* acc = reinterpret_cast<float*>(smem + STAGES * STAGE);
  uint8_t* tables = smem + STAGES * STAGE + Cfg<NT>::ACC_BYTES;
  const Tables tb = {reinterpret_cast<uint16_t*>(tables), reinterpret_cast<uint16_t*>(tables + kSlots),
                     reinterpret_cast<float*>(tables + kSlots + kIdx)};
  int* err = reinterpret_cast<int*>(p.header);
  const int cta = (int)blockIdx.x, n_cta = (int)gridDim.x, T = (int)D.T;   // T < n_cta
  setup<NT, STAGES>(b, warp);
  const uint32_t epoch = *reinterpret_cast<volatile uint32_t*>(p.header + 1) + 1;

  const uint32_t tag = 1 + epoch % kTagMask;
  const bool scores = p.a.logits_in == nullptr && cta < p.s.n_slab;
  Plan plan(D, cta, n_cta);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (scores) gate_wait();
    if (lane == 0) {
      Ring<STAGES> ring;
      int64_t loaded = 0;
      bool ok = true;
      // the token rows of an output block, into stage q
      auto rows = [&](const Ring<STAGES>& q, const Blocks& k) {
        tma2d(smem_base + q.stage * STAGE + A_BYTES, k.shared ? &p.hs : &p.h, smem_u32(&b.full[q.stage]), k.at * BK,
              k.slot * NT);
      };
#pragma unroll 1
      for (int r = D.S > 0 ? SHARED : HIDDEN; ok && r <= OUTPUT; ++r) {
        if (r == HIDDEN) {
          ok = bar_wait(&b.list, 0, &b.abort, err);
          if (!ok) break;
          plan.select(s_active);
        }
        Run run = plan.run(r), tokens = run;
        // The output's weights are loaded at once, its tokens' hidden rows when every CTA has written
        // its own: `ahead` stages, from `behind` on, lack them.
        bool have_rows = r != OUTPUT;
        Ring<STAGES> behind = ring;
        int ahead = 0;
        auto wait_rows = [&]() {
          ok = ok && word_wait(p.header + ROWS, (uint32_t)n_cta + p.a.absent, &b.abort, err);
          asm volatile("fence.proxy.async;" ::: "memory");   // generic writes of other CTAs, read by TMA
          have_rows = true;
          // the same blocks again, from the run's start. Also when the launch has failed: a stage that
          // lacked its rows would never be full, and drain() would wait its whole limit for each
          while (ahead > 0 && tokens.next()) {
            Blocks k(plan, tokens.s.k0);
            for (int kb = tokens.s.k0; kb < tokens.s.k1 && ahead > 0; ++kb, --ahead) {
              rows(behind, k);
              behind.step();
              k.step(plan);
            }
          }
        };
        // the next stage, or false
        auto acquire = [&]() {
          if (loaded == SLAB0 && scores)   // the ring's last stages hold W_r first
            ok = ok && bar_wait(&b.slab_free, 0, &b.abort, err);
          ok = ok && bar_wait(&b.empty[ring.stage], ring.phase ^ 1u, &b.abort, err);
          if (ok) mbar_arrive_expect_tx(smem_u32(&b.full[ring.stage]), STAGE);
          return ok;
        };
#pragma unroll 1
        while (ok && run.next()) {
          if (r != OUTPUT) {   // 64 gate and the 64 up rows beside them
            const int per = r == SHARED ? plan.per_s : plan.per_h, f = r == SHARED ? D.f_s : D.f;
            const int tile = (int)run.s.t, slot = tile / per, j0 = (tile - slot * per) * 64;
            const int e = r == SHARED ? slot : tb.slots[slot];
            const CUtensorMap* m = r == SHARED ? &p.ws13 : &p.w13;
#pragma unroll 1
            for (int kb = run.s.k0; kb < run.s.k1 && acquire(); ++kb) {
              const uint32_t a_s = smem_base + ring.stage * STAGE, bar = smem_u32(&b.full[ring.stage]);
              tma3d(a_s, m, bar, kb * BK, j0, e);
              tma3d(a_s + A_BYTES / 2, m, bar, kb * BK, f + j0, e);
              tma2d(a_s + A_BYTES, &p.x, bar, kb * BK, 0);
              ring.step();
              ++loaded;
            }
          } else {
            Blocks k(plan, run.s.k0);
            const int n0 = (int)run.s.t * BM;
#pragma unroll 1
            for (int kb = run.s.k0; kb < run.s.k1; ++kb) {
              if (!have_rows && ahead == STAGES) wait_rows();   // the ring is full of weights
              if (!acquire()) break;
              tma3d(smem_base + ring.stage * STAGE, k.shared ? &p.ws2 : &p.w2, smem_u32(&b.full[ring.stage]), k.at * BK, n0,
                    k.shared ? k.slot : tb.slots[k.slot]);
              if (have_rows) rows(ring, k);
              else ++ahead;
              ring.step();
              ++loaded;
              k.step(plan);
            }
          }
        }
        if (!have_rows && ahead > 0) wait_rows();
      }
      drain<STAGES>(b, ring, loaded, err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    Ring<STAGES> ring;
    int it = 0;
    bool ok = true;
    const bool one = elect_one();
#pragma unroll 1
    for (int r = D.S > 0 ? SHARED : HIDDEN; ok && r <= OUTPUT; ++r) {
      if (r == HIDDEN) {
        ok = warp_bar_wait(smem_u32(&b.list), 0, &b.abort, err);
        if (!ok) break;
        plan.select(s_active);
      }
      ok = mma_run<NT, STAGES>(b, smem_base, plan.run(r), ring, it, one, err);
    }
    if (one) {
      umma1_commit(smem_u32(&b.final));   // every MMA retired before the tensor memory is released
      bar_wait(&b.final, 0, nullptr, err);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ scores, selection, results
    int it = 0;
    bool ok = true;
    // the bias waits in the table of gates, which is filled later (read when it is needed, it would
    // come from HBM behind the stream)
    if (cta < T && p.a.bias != nullptr) copy_floats(tb.gate, p.a.bias, D.E, D.E % 4 == 0);
    if (scores) {
      partial_scores<NT, __nv_bfloat16, true>(p.s, cta, acc, reinterpret_cast<float*>(smem + SLAB0 * STAGE), (STAGES - SLAB0) * STAGE / 4);
      __threadfence();
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the stages become the TMA's again
      ct_sync();
      if (threadIdx.x == 64) {
        add_release(p.header + SCORES, 1u);
        mbar_arrive(smem_u32(&b.slab_free));
      }
    }
    if (cta < T) {
      if (p.a.logits_in == nullptr) {
        if (threadIdx.x == 64) ok = word_wait(p.header + SCORES, (uint32_t)p.s.n_slab, &b.abort, err);
        ok = !ct_any(!ok);
      }
      if (ok)
        select_experts(p.s, cta, reinterpret_cast<float*>(smem), STAGES * STAGE / 4, acc + kMaxE,
                       reinterpret_cast<uint32_t*>(acc), s_top, tb.gate, tag);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the ring held partial scores
      ct_sync();
    }
    Finish<NT> f{p, tb, plan, s_wt, 0};
#pragma unroll 1
    for (int r = D.S > 0 ? SHARED : HIDDEN; ok && r <= OUTPUT; ++r) {
      if (r == HIDDEN) {
        const int active = build_tables(p.s, tb, tag, s_bits, &s_active, &b.abort, err);
        ok = active > 0;
        if (!ok) break;
        plan.select(active);
        if (threadIdx.x == 64) mbar_arrive(smem_u32(&b.list));
      }
      f.r = r;
      ok = take_run<NT>(b, plan.run(r), it, r == SHARED ? cta - T : cta, p.flags + r * n_cta, epoch,
                        p.part + (int64_t)r * n_cta * NT * BM, acc, err, f, NT > 16 && r == OUTPUT && plan.tiles_out * kScatter <= n_cta);
      if (ok && r == HIDDEN) {
        // this CTA's hidden rows are written, for the TMA of any CTA
        __threadfence();
        asm volatile("fence.proxy.async;" ::: "memory");
        ct_sync();
        if (threadIdx.x == 64) add_release(p.header + ROWS, 1u);
      }
    }
  }
  teardown<NT>(b, warp);
  // the tags start again after this launch: no word may still hold one
  if (leave(p.header, epoch) && tag == kTagMask)
    for (int i = 0; i < kDecodeMaxT * kMaxK; ++i) p.s.chosen[i] = 0;
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
  if (num_sms <= kDecodeMaxT) return MOE_ERR_UNSUPPORTED_DEVICE;
  DecodeTc p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.s = select_args(a, num_sms);
  p.header = reinterpret_cast<uint32_t*>(a.ws);
  p.flags = p.header + 256;
  p.part = reinterpret_cast<float*>(a.ws + a.L.part);
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
