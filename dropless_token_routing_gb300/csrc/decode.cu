// The whole MoE layer for a few tokens in fp32, in one cooperative launch on the FMA pipes (the
// fp32 workloads are small: the launch's chain of steps is what they cost, not their bytes).
//
// Scores, selection and tables as in the bf16 layer (decode_select.cuh). Then the warps divide the
// hidden rows evenly: an item is two of them (each a gate row and an up row of W13) with up to four
// of the tokens that selected the expert, so that many tokens make more items, not longer ones.
// After a grid barrier the CTAs divide the output: four rows of W2 and four tokens, whose experts
// (those that any of them selected and the shared ones) the warps divide; no expert's result is
// ever written.
//
// Nothing is rounded below fp32. Bound by the chain's latency: T = 1, d = 512: 3.2 MB in 18 us (45 us as
// a chain of launches); T = 59, d = 296, 25 experts, top-7: 70 us.
#include <string.h>

#include <mutex>

#include "decode_select.cuh"
#include "trace.h"

namespace moe {
namespace {

using namespace decode;

constexpr int kBuf = 16384;        // floats of a slab of W_r, and of partial scores
constexpr int GROUP = 4;           // tokens that share a pass over weight rows
constexpr int HR = 2, OR = 4;      // hidden rows (pairs of W13's) and output rows of an item
constexpr int FT = 512;            // threads; the last CT of them select

struct DecodeF32 {
  DecodeArgs a;
  Select s;
  float *h, *hs;                   // [slot][T][f], [S][T][f_s]
};

template <int NT> constexpr int smem_floats() { return kBuf + RT * NT + kMaxE + CT + (kExtra + 3) / 4 + kMaxE + 1 + kMaxE / 2; }

__device__ __forceinline__ float dot4(const float4& a, const float4& b, float s) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, s))));
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Up to GROUP tokens, n of them, and their gates (the same in all lanes).
struct Group {
  int n, t[GROUP];
  float w[GROUP];
};
// Tokens GROUP * g .. of those that selected expert e, in token order.
__device__ __forceinline__ Group routed_group(const Tables& tb, int e, int g, int T, int k, int lane) {
  float g0 = 0.f, g1 = 0.f;   // gates of tokens lane and lane + 32
  bool in0 = false, in1 = false;
  for (int j = 0; j < k; ++j) {
    if (lane < T && tb.idx[lane * k + j] == e) {
      in0 = true;
      g0 = tb.gate[lane * k + j];
    }
    if (lane + 32 < T && tb.idx[(lane + 32) * k + j] == e) {
      in1 = true;
      g1 = tb.gate[(lane + 32) * k + j];
    }
  }
  const uint32_t lo = __ballot_sync(0xffffffffu, in0), hi = __ballot_sync(0xffffffffu, in1);
  uint64_t mask = lo | (uint64_t)hi << 32;
  for (int i = 0; i < g * GROUP; ++i) mask &= mask - 1;
  Group r;
  r.n = 0;
#pragma unroll
  for (int i = 0; i < GROUP; ++i) {
    const bool some = mask != 0;
    const int t = some ? __ffsll((long long)mask) - 1 : 0;
    mask &= mask - 1;   // 0 stays 0
    const float w = __shfl_sync(0xffffffffu, t < 32 ? g0 : g1, t & 31);
    r.t[i] = t;
    r.w[i] = w;
    r.n += some ? 1 : 0;
  }
  return r;
}

// Hidden rows j .. j + HR - 1 of one expert for a group: h[t * f + j] = gate * silu(w1 . x_t) * (w3 . x_t).
__device__ __forceinline__ void hidden_rows(const float* __restrict__ w1, const float* __restrict__ w3, const float* x, int d,
                                            const Group& r, float* h, int f, int j, int lane) {
  float g[HR][GROUP] = {}, u[HR][GROUP] = {};
#pragma unroll 2
  for (int i = lane * 4; i < d; i += 128) {
    float4 a[HR], b[HR];
#pragma unroll
    for (int o = 0; o < HR; ++o) {
      a[o] = __ldg(reinterpret_cast<const float4*>(w1 + (int64_t)o * d + i));
      b[o] = __ldg(reinterpret_cast<const float4*>(w3 + (int64_t)o * d + i));
    }
#pragma unroll
    for (int q = 0; q < GROUP; ++q) {
      if (q >= r.n) break;
      const float4 v = *reinterpret_cast<const float4*>(x + (int64_t)r.t[q] * d + i);   // y may be x's buffer
#pragma unroll
      for (int o = 0; o < HR; ++o) {
        g[o][q] = dot4(a[o], v, g[o][q]);
        u[o][q] = dot4(b[o], v, u[o][q]);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < GROUP; ++q) {
    if (q >= r.n) break;
#pragma unroll
    for (int o = 0; o < HR; ++o) {
      const float gs = warp_sum(g[o][q]), us = warp_sum(u[o][q]);
      if (lane == 0) __stcg(h + (int64_t)r.t[q] * f + j + o, r.w[q] * (silu_f(gs) * us));
    }
  }
}

// y[o] += W2's row o of w (rows f apart) . h of the group's tokens (bit q of `in`: token q takes
// part). h was written in this launch, but no SM reads it before the grid barrier: L1 holds none.
__device__ __forceinline__ void output_rows(const float* __restrict__ w, const float* h, int f, uint32_t in, float (&y)[OR][GROUP],
                                            int lane) {
#pragma unroll 2
  for (int i = lane * 4; i < f; i += 128) {
    float4 a[OR];
#pragma unroll
    for (int o = 0; o < OR; ++o) a[o] = __ldg(reinterpret_cast<const float4*>(w + (int64_t)o * f + i));
#pragma unroll
    for (int q = 0; q < GROUP; ++q)
      if (in >> q & 1u) {
        const float4 v = *reinterpret_cast<const float4*>(h + (int64_t)q * f + i);
#pragma unroll
        for (int o = 0; o < OR; ++o) y[o][q] = dot4(a[o], v, y[o][q]);
      }
  }
}

template <int NT>
__global__ void __launch_bounds__(FT, 1) decode_f32_kernel(const __grid_constant__ DecodeF32 p) {
  extern __shared__ __align__(16) float smem[];
  __shared__ uint32_t s_bits[kMaxE / 32], s_top[2 * kMaxK];
  __shared__ int s_active, s_entries, s_list[GROUP * kMaxK + kMaxShared];
  __shared__ float s_part[2][FT / 32][GROUP * OR];
  __shared__ volatile int s_abort;
  const moe_dims& D = p.a.dm;
  const int T = (int)D.T, k = D.k, d = D.d, lane = threadIdx.x & 31;
  const int cta = (int)blockIdx.x, n_cta = (int)gridDim.x;   // T < n_cta
  float *buf = smem, *xs = buf + kBuf, *keys = xs + RT * NT, *tmp = keys + kMaxE;
  uint8_t* tables = reinterpret_cast<uint8_t*>(tmp + CT);
  const Tables tb = {reinterpret_cast<uint16_t*>(tables), reinterpret_cast<uint16_t*>(tables + kSlots),
                     reinterpret_cast<float*>(tables + kSlots + kIdx)};
  int* groups = reinterpret_cast<int*>(tables + kExtra);          // groups of the slots before each slot
  uint16_t* slot_of = reinterpret_cast<uint16_t*>(groups + kMaxE + 1);
  uint32_t* header = p.s.header;
  int* err = reinterpret_cast<int*>(header);
  if (threadIdx.x == 0) {
    s_abort = 0;
    s_active = 0;
  }
  __syncthreads();
  const uint32_t epoch = *reinterpret_cast<volatile uint32_t*>(header + 1) + 1, tag = 1 + epoch % kTagMask;

  if (threadIdx.x >= FT - CT) {
    bool ok = true;
    const bool first = ct_tid() == 0;
    if (cta < T && p.a.bias != nullptr) copy_floats(tb.gate, p.a.bias, D.E, D.E % 4 == 0);
    if (p.a.logits_in == nullptr && cta < p.s.n_slab) {
      partial_scores<NT, float, false>(p.s, cta, xs, buf, kBuf);
      __threadfence();
      ct_sync();
      if (first) add_release(header + SCORES, 1u);
    }
    if (cta < T) {
      if (p.a.logits_in == nullptr) {
        if (first) ok = word_wait(header + SCORES, (uint32_t)p.s.n_slab, &s_abort, err);
        ok = !ct_any(!ok);
      }
      if (ok) select_experts(p.s, cta, buf, kBuf, tmp, reinterpret_cast<uint32_t*>(keys), s_top, tb.gate, tag);
      ct_sync();
    }
    if (ok) {
      const int active = build_tables(p.s, tb, tag, s_bits, &s_active, &s_abort, err);
      // groups of each slot: its tokens, counted in `keys`, in fours
      int* count = reinterpret_cast<int*>(keys);
      for (int i = ct_tid(); i < active; i += CT) {
        slot_of[tb.slots[i]] = (uint16_t)i;
        count[tb.slots[i]] = 0;
      }
      ct_sync();
      for (int i = ct_tid(); i < T * k; i += CT) atomicAdd(count + tb.idx[i], 1);
      ct_sync();
      if (ct_tid() < 32) {
        int sum = 0;
        for (int s0 = 0; s0 < active; s0 += 32) {
          const int g = s0 + lane < active ? (count[tb.slots[s0 + lane]] + GROUP - 1) / GROUP : 0;
          int inc = g;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
          }
          if (s0 + lane < active) groups[s0 + lane] = sum + inc - g;
          sum += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) groups[active] = sum;
      }
    }
  }
  __syncthreads();
  const int active = s_active;   // 0: the wait for the selection ran out
  if (active > 0) {
    const int warps = n_cta * (FT / 32), warp = cta * (FT / 32) + (int)(threadIdx.x >> 5);
    const float* x = static_cast<const float*>(p.a.x);
    const int g_all = (T + GROUP - 1) / GROUP;   // groups of all tokens
    // items: (slot, group, row) of the selected experts, then (shared expert, group, row)
    const int64_t routed = (int64_t)groups[active] * (D.f / HR), items = routed + (int64_t)D.S * g_all * (D.f_s / HR);
    const int64_t i0 = items * warp / warps, i1 = items * (warp + 1) / warps;
    int64_t seen = -1;   // the group that `r` holds
    int slot = 0;
    Group r;
    for (int64_t i = i0; i < i1; ++i) {
      const bool sh = i >= routed;
      const int f = sh ? D.f_s : D.f;
      const int64_t at = sh ? i - routed : i, g = at / (f / HR);
      const int j = (int)(at - g * (f / HR)) * HR;
      if (!sh) {
        if (seen != g) {
          while (groups[slot + 1] <= (int)g) ++slot;
          r = routed_group(tb, tb.slots[slot], (int)g - groups[slot], T, k, lane);
          seen = g;
        }
        const float* w = static_cast<const float*>(p.a.w13) + ((int64_t)tb.slots[slot] * 2 * f + j) * d;
        hidden_rows(w, w + (int64_t)f * d, x, d, r, p.h + (int64_t)slot * T * f, f, j, lane);
      } else {
        const int s = (int)(g / g_all), t0 = (int)(g - (int64_t)s * g_all) * GROUP;
        r.n = min(GROUP, T - t0);
#pragma unroll
        for (int q = 0; q < GROUP; ++q) {
          r.t[q] = min(t0 + q, T - 1);
          r.w[q] = 1.f;
        }
        const float* w = static_cast<const float*>(p.a.ws13) + ((int64_t)s * 2 * f + j) * d;
        hidden_rows(w, w + (int64_t)f * d, x, d, r, p.hs + (int64_t)s * T * f, f, j, lane);
      }
    }
    __threadfence();
    __syncthreads();
    bool ok = true;
    if (threadIdx.x == 0) {
      add_release(header + ROWS, 1u);
      ok = word_wait(header + ROWS, (uint32_t)n_cta + p.a.absent, &s_abort, err);
    }
    ok = !__syncthreads_or(!ok);
    if (ok) {
      // items of a whole CTA, whose warps divide the experts: few tokens leave few items, and an
      // expert after the other costs a latency each
      const int64_t out = (int64_t)(d / OR) * g_all, o0 = out * cta / n_cta, o1 = out * (cta + 1) / n_cta;
      const int w = (int)(threadIdx.x >> 5);
      int have = -1, buf_at = 0;
      for (int64_t i = o0; i < o1; ++i, buf_at ^= 1) {
        const int g = (int)(i / (d / OR)), n = (int)(i - (int64_t)g * (d / OR)) * OR, t0 = g * GROUP;
        if (g != have) {   // the group's experts: (slot << GROUP | tokens), then the shared ones
          have = g;
          __syncthreads();
          if (w == 0) {
            uint32_t in[GROUP], any = 0;   // lane l: bit b: token t0 + q selected slot 32 l + b
#pragma unroll
            for (int q = 0; q < GROUP; ++q) {
              in[q] = 0;
              if (t0 + q < T)
                for (int j = 0; j < k; ++j) {
                  const int s = slot_of[tb.idx[(t0 + q) * k + j]];   // the same in all lanes
                  if (s >> 5 == lane) in[q] |= 1u << (s & 31);
                }
              any |= in[q];
            }
            const int c = __popc(any);
            int inc = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int v = __shfl_up_sync(0xffffffffu, inc, o);
              if (lane >= o) inc += v;
            }
            int at = inc - c;
            for (uint32_t bits = any; bits != 0; bits &= bits - 1) {
              const int bit = __ffs((int)bits) - 1;
              s_list[at++] = (lane * 32 + bit) << GROUP | (in[0] >> bit & 1) | (in[1] >> bit & 1) << 1 | (in[2] >> bit & 1) << 2 |
                             (in[3] >> bit & 1) << 3;
            }
            const int routed_n = __shfl_sync(0xffffffffu, inc, 31);
            if (lane < D.S) s_list[routed_n + lane] = (kMaxE + lane) << GROUP | ((1 << min(GROUP, T - t0)) - 1);
            if (lane == 0) s_entries = routed_n + D.S;
          }
          __syncthreads();
        }
        float y[OR][GROUP] = {};
        for (int e = w; e < s_entries; e += FT / 32) {
          const int entry = s_list[e], s = entry >> GROUP, m = entry & ((1 << GROUP) - 1);
          if (s < kMaxE)
            output_rows(static_cast<const float*>(p.a.w2) + ((int64_t)tb.slots[s] * d + n) * D.f, p.h + ((int64_t)s * T + t0) * D.f,
                        D.f, m, y, lane);
          else
            output_rows(static_cast<const float*>(p.a.ws2) + ((int64_t)(s - kMaxE) * d + n) * D.f_s,
                        p.hs + ((int64_t)(s - kMaxE) * T + t0) * D.f_s, D.f_s, m, y, lane);
        }
        if (w < s_entries) {
#pragma unroll
          for (int q = 0; q < GROUP; ++q)
#pragma unroll
            for (int o = 0; o < OR; ++o) {
              const float v = warp_sum(y[o][q]);
              if (lane == q * OR + o) s_part[buf_at][w][lane] = v;
            }
        }
        __syncthreads();
        if (threadIdx.x < GROUP * OR) {   // a token's row: the warps' parts in their order
          const int q = threadIdx.x / OR, o = threadIdx.x % OR;
          if (t0 + q < T) {
            float v = 0.f;
            for (int e = 0; e < min(s_entries, FT / 32); ++e) v += s_part[buf_at][e][threadIdx.x];
            const int64_t at = (int64_t)(t0 + q) * d + n + o;
            if (p.a.residual != nullptr) v += static_cast<const float*>(p.a.residual)[at];   // may be y's own buffer
            static_cast<float*>(p.a.y)[at] = v;
          }
        }
      }
    }
  }
  __syncthreads();
  if (leave(header, epoch) && tag == kTagMask)   // the tags start again after this launch
    for (int i = 0; i < kDecodeMaxT * kMaxK; ++i) p.s.chosen[i] = 0;
}

template <int NT>
int launch_nt(const DecodeF32& p, int num_sms, cudaStream_t st) {
  constexpr int SMEM = smem_floats<NT>() * 4;
  static std::mutex mu;   // per device, once: the shared-memory attribute
  static bool attr_set[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MOE_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!attr_set[dev]) {
      if (cudaFuncSetAttribute(decode_f32_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess)
        return MOE_ERR_CUDA;
      attr_set[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_sms);
  cfg.blockDim = dim3(FT);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;   // the CTAs wait on one another
  at[0].val.cooperative = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  TraceScope ts(TP_DECODE, st);
  return cudaLaunchKernelEx(&cfg, decode_f32_kernel<NT>, p) == cudaSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // namespace

int launch_decode_simt(const DecodeArgs& a, int num_sms, cudaStream_t st) {
  if (num_sms > kMaxStreamCtas) num_sms = kMaxStreamCtas;
  if (num_sms <= kDecodeMaxT) return MOE_ERR_UNSUPPORTED_DEVICE;
  DecodeF32 p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.s = select_args(a, num_sms);
  p.h = reinterpret_cast<float*>(a.ws + a.L.h);
  p.hs = reinterpret_cast<float*>(a.ws + a.L.hs);
  return a.dm.T <= 16 ? launch_nt<16>(p, num_sms, st) : launch_nt<64>(p, num_sms, st);
}

}  // namespace moe
