// Scores, selection and tables of the few-token layer, for its bf16 kernel (decode_tc.cu) and its
// fp32 one (decode.cu). They run on CT threads of a block, its last ones.
//
// CTA c takes a slab of W_r's rows and leaves the slab's scores in the workspace; CTA t sums token
// t's in their order, ranks the experts and writes the selection; every CTA then builds the list of
// selected experts.
#pragma once

#include "stream.cuh"

namespace moe {
namespace decode {

using namespace stream;

constexpr int RT = 128;            // rows of W_r that a CTA takes at a time
// tables: selected experts, and the tokens' selections
constexpr int kSlots = kMaxE * 2;                       // uint16 expert of each slot
constexpr int kIdx = kDecodeMaxT * kMaxK * 2;           // uint16 [T][k]
constexpr int kGate = kDecodeMaxT * kMaxK * 4;          // fp32 [T][k]; first the bias
static_assert(kGate >= kMaxE * 4, "the bias waits in the table of gates");
constexpr int kExtra = kSlots + kIdx + kGate;

struct Select {
  moe_dims dm;
  const void* x;
  const float *w_r, *bias, *logits_in;
  int32_t* idx_out;
  float* gate_out;
  int n_slab, slab;      // CTAs that take a slab of W_r, rows of each
  uint32_t* header;      // error, epoch, leave count, counters (enum)
  float* score_part;     // [T][n_slab][E]
  uint64_t* chosen;      // [T][k] selections
};

enum Counter { SCORES = 3, ROWS };   // words of the header
// A selection is one 64-bit word: gate (32 bits), expert (kTagShift bits) and the launch's tag
// (22 bits, from the epoch, never 0). The words are cleared before the tags start again.
constexpr int kTagShift = 10;
constexpr uint32_t kTagMask = (1u << (32 - kTagShift)) - 1;
static_assert(kMaxE == 1 << kTagShift, "");

struct Tables {
  uint16_t* slots;
  uint16_t* idx;
  float* gate;
};

// ------------------------------------------------------------------ scores and selection
__device__ __forceinline__ void gate_open() { asm volatile("bar.arrive 2, 288;" ::: "memory"); }
__device__ __forceinline__ void gate_wait() { asm volatile("bar.sync 2, 288;" ::: "memory"); }

// `n` floats global -> shared by the result warps, 16 bytes at a time where both ends allow.
__device__ __forceinline__ void copy_floats(float* dst, const float* src, int n, bool vec) {
  const int tid = ct_tid();
  if (vec) {
#pragma unroll 4
    for (int i = tid * 4; i < n; i += CT * 4) cp_async16(smem_u32(dst + i), src + i);
  } else {
#pragma unroll 4
    for (int i = tid; i < n; i += CT)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst + i)), "l"(src + i) : "memory");
  }
}
__device__ __forceinline__ void copies_landed() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  ct_sync();
}

// Partial scores of this CTA's slab. xs: [rows][NT] floats, ws: `cap` floats of shared memory (in the
// bf16 layer stages of the ring that the producer leaves alone until slab_free). The first part of W_r is asked for before anything
// else: behind the weight stream's loads it would wait for all of those, so the producer starts
// once it is on its way (gate_open, GATE). W_r goes through shared memory, not registers: the loop
// stays a few instructions long (unrolled over 64 register loads it took 8 us, most of it
// instruction fetches).
template <int NT, typename T_, bool GATE>
__device__ __forceinline__ void partial_scores(const Select& p, int cta, float* xs, float* ws, int cap) {
  constexpr int TS = 8;   // tokens at a time in registers
  const moe_dims& D = p.dm;
  const int T = (int)D.T, E = D.E, d = D.d, tid = ct_tid();
  const int d0 = cta * p.slab, d1 = min(d, d0 + p.slab);
  const T_* x = static_cast<const T_*>(p.x);
  const int at_once = min(RT, cap / E);   // rows of W_r
  for (int r0 = d0; r0 < d1; r0 += at_once) {
    const int n = min(at_once, d1 - r0);
    copy_floats(ws, p.w_r + (int64_t)r0 * E, n * E, E % 4 == 0);
    if (GATE && r0 == d0) gate_open();
    for (int i = tid; i < n * NT; i += CT) {
      const int t = i / n, r = i - t * n;
      xs[r * NT + t] = t < T ? to_f32(x[(int64_t)t * d + r0 + r]) : 0.f;
    }
    copies_landed();
    // one expert and TS tokens at a time
#pragma unroll 1
    for (int i = tid; i < E * ((T + TS - 1) / TS); i += CT) {
      const int e = i % E, t0 = i / E * TS;
      float* out = p.score_part + ((int64_t)t0 * p.n_slab + cta) * E + e;
      float s[TS];
#pragma unroll
      for (int t = 0; t < TS; ++t) s[t] = r0 > d0 && t0 + t < T ? __ldcg(out + (int64_t)t * p.n_slab * E) : 0.f;
#pragma unroll 4
      for (int r = 0; r < n; ++r) {
        const float w = ws[r * E + e];
        const float4* xr = reinterpret_cast<const float4*>(xs + r * NT + t0);
#pragma unroll
        for (int t = 0; t < TS; t += 4) {
          const float4 v = xr[t / 4];
          s[t] = fmaf(v.x, w, s[t]);
          s[t + 1] = fmaf(v.y, w, s[t + 1]);
          s[t + 2] = fmaf(v.z, w, s[t + 2]);
          s[t + 3] = fmaf(v.w, w, s[t + 3]);
        }
      }
#pragma unroll
      for (int t = 0; t < TS; ++t)
        if (t0 + t < T) __stcg(out + (int64_t)t * p.n_slab * E, s[t]);
    }
    ct_sync();
  }
}

// Order-preserving map of a float to uint32, above 0 for every finite one; NaN is ranked last.
__device__ __forceinline__ uint32_t rank_key(float x) {
  if (!(x == x)) return 1u;
  const uint32_t u = __float_as_uint(x + 0.f);   // -0 ranks as +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// Token t's scores, ranked. Shared memory: buf [cap] floats (the ring, idle in a CTA with a token),
// through which the partial rows come, all of them in flight; tmp [CT]; keys [E], a multiple of 4
// readable; top [2 * kMaxK]; bias [E].
// An expert's rank is the number of experts before it (larger key, or the same and a lower index),
// which every thread counts for its own: no rounds over k. All loops are short on purpose: this is
// code that a CTA runs once, and fetching it is what it costs.
__device__ __forceinline__ void select_experts(const Select& p, int t, float* buf, int cap, float* tmp, uint32_t* keys,
                                               uint32_t* top, const float* bias, uint32_t tag) {
  const moe_dims& D = p.dm;
  const int E = D.E, k = D.k, tid = ct_tid();
  const bool given = p.logits_in != nullptr;
  const int rows = given ? 1 : p.n_slab, at_once = cap / E;
  const float* in = given ? p.logits_in + (int64_t)t * E : p.score_part + (int64_t)t * rows * E;
  for (int i = tid; i < ((E + 3) & ~3); i += CT) keys[i] = 0u;
  for (int r0 = 0; r0 < rows; r0 += at_once) {
    const int n = min(at_once, rows - r0);
    copy_floats(buf, in + (int64_t)r0 * E, n * E, E % 4 == 0);
    copies_landed();
#pragma unroll 1
    for (int e0 = 0; e0 < E; e0 += CT) {
      // ng threads share a column, each summing every ng-th row
      const int cols = min(E - e0, CT), ng = CT / cols, g = tid / cols, c = e0 + tid % cols;
      float s = 0.f;
      if (g < ng) {
#pragma unroll 4
        for (int r = g; r < n; r += ng) s += buf[r * E + c];
      }
      tmp[tid] = s;
      ct_sync();
      if (tid < cols) {
        for (int i = cols; i < ng * cols; i += cols) s += tmp[tid + i];
        if (r0 > 0) s += __uint_as_float(keys[c]);   // the sum so far
        if (r0 + n < rows) keys[c] = __float_as_uint(s);
        else keys[c] = rank_key(p.bias != nullptr ? s + bias[c] : s);   // one fp32 rounding
      }
      ct_sync();
    }
  }
#pragma unroll 1
  for (int e = tid; e < E; e += CT) {
    const uint32_t key = keys[e];
    int rank = 0;
#pragma unroll 2
    for (int i = 0; i < E; i += 4) {   // keys past E are 0, below every other
      const uint4 v = *reinterpret_cast<const uint4*>(keys + i);
      rank += (v.x > key || (v.x == key && i < e)) + (v.y > key || (v.y == key && i + 1 < e)) +
              (v.z > key || (v.z == key && i + 2 < e)) + (v.w > key || (v.w == key && i + 3 < e));
    }
    if (rank < k) {
      top[rank] = e;
      top[kMaxK + rank] = key;
    }
  }
  ct_sync();
  if (tid < 32) {
    const float v = key_value(top[kMaxK + min(tid, k - 1)]);
    const float largest = __shfl_sync(0xffffffffu, v, 0);   // by all lanes
    float w = tid < k ? expf(v - largest) : 0.f, sum = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w /= sum;
    if (tid < k) {
      const int64_t q = (int64_t)t * k + tid;
      const int32_t e = (int32_t)top[tid];
      // expert, gate and the launch in one word: whoever reads it needs no other signal
      asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p.chosen + q),
                   "l"((uint64_t)(tag << kTagShift | (uint32_t)e) << 32 | __float_as_uint(w))
                   : "memory");
      if (p.idx_out != nullptr) p.idx_out[q] = e;
      if (p.gate_out != nullptr) p.gate_out[q] = w;
    }
  }
}

// The selected experts in ascending order, and the tokens' selections, once they are all there
// (their words carry this launch's tag). Returns their number, 0 when the wait ran out.
// bits: kMaxE / 32 words, count: one int of shared memory.
__device__ __forceinline__ int build_tables(const Select& p, const Tables& tb, uint32_t tag, uint32_t* bits, int* count,
                                            volatile int* abort, int* err) {
  const moe_dims& D = p.dm;
  const int n = (int)D.T * D.k, tid = ct_tid();
  if (tid < kMaxE / 32) bits[tid] = 0u;
  ct_sync();
  const uint64_t t0 = global_ns();
  bool ok = true;
#pragma unroll 1
  for (int i = tid; ok && i < n; i += CT) {
    uint64_t w;
    while (true) {
      asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(w) : "l"(p.chosen + i) : "memory");
      if ((uint32_t)(w >> (32 + kTagShift)) == tag) break;
      if (*abort || global_ns() - t0 > kWaitLimitNs) {
        if (!*abort) record_error(err, MOE_ERR_DEVICE_TIMEOUT);
        *abort = 1;
        ok = false;
        break;
      }
    }
    if (!ok) break;
    const int e = (int)(w >> 32) & (kMaxE - 1);
    tb.idx[i] = (uint16_t)e;
    tb.gate[i] = __uint_as_float((uint32_t)w);
    atomicOr(bits + (e >> 5), 1u << (e & 31));
  }
  if (ct_any(!ok)) return 0;
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

// The select part of a launch (host).
inline Select select_args(const DecodeArgs& a, int num_sms) {
  Select s = {};
  s.dm = a.dm;
  s.x = a.x;
  s.w_r = a.w_r;
  s.bias = a.bias;
  s.logits_in = a.logits_in;
  s.idx_out = a.idx_out;
  s.gate_out = a.gate_out;
  // slabs of at least 8 rows of W_r
  s.slab = (a.dm.d + num_sms - 1) / num_sms;
  if (s.slab < 8) s.slab = 8;
  s.n_slab = (a.dm.d + s.slab - 1) / s.slab;
  s.header = reinterpret_cast<uint32_t*>(a.ws);
  s.score_part = reinterpret_cast<float*>(a.ws + a.L.score_part);
  s.chosen = reinterpret_cast<uint64_t*>(a.ws + kOpFlags);
  return s;
}

}  // namespace decode
}  // namespace moe
