// Host-side internals of the few-token operators: workspace layouts and kernel launchers.
#pragma once

#include "internal.h"

namespace moe {

constexpr size_t kOpFlags = 8192;     // error word, launch counters, and from byte 1024 flags
constexpr size_t kOpHeader = kOpFlags + 8 * 64 * kMaxK;   // and the selections of 64 tokens
constexpr int kDecodeMaxT = 64;       // tokens of moe_layer_decode
static_assert(kOpHeader == kOpFlags + 8 * kDecodeMaxT * kMaxK, "");

constexpr int64_t kMaxLd = 1ll << 36;   // elements between rows
inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int kMaxStreamCtas = 160;   // CTAs of a weight stream
constexpr int kMinStreamRun = 2;      // K blocks of a CTA's run (1, 2, 4: the same within 2 %, 22 us with d = 320)
constexpr int kWholeTiles = 16;       // K blocks that a join costs (6, 16: 42, 40 us with 19 tokens, d = 2112; 0: 45)

// ------------------------------------------------------------------ decode
constexpr int kDecodeRuns = 3;   // shared, hidden, output
struct DecodeLayout {
  size_t score_part; // [T][slabs][E] fp32 partial scores
  size_t part;       // bf16: [kDecodeRuns + 1][CTA][token columns][128] fp32 partial tiles
  // hidden rows times their gates: fp32 [slot][T][f] and [S][T][f_s]; bf16 [slot][token columns][f]
  // and [S][token columns][f_s]
  size_t h, hs;
  size_t total;
};
DecodeLayout decode_layout(const moe_dims& d);

struct DecodeArgs {
  const void *x, *residual;
  const float *w_r, *bias, *logits_in;
  const void *w13, *w2, *ws13, *ws2;
  int32_t* idx_out;
  float* gate_out;
  void* y;
  uint8_t* ws;
  uint32_t absent;   // CTAs beyond the launch's that the hidden rows are waited for: 0, 1 lets the wait run out
  DecodeLayout L;
  moe_dims dm;
};
int decode_token_columns(int64_t T);   // MMA columns that T tokens take
// slots of the hidden rows: experts that T tokens can select
inline int64_t decode_slots(const moe_dims& d) { return d.T * d.k < d.E ? d.T * d.k : d.E; }
int launch_decode_tc(const DecodeArgs& a, int num_sms, cudaStream_t st);
int launch_decode_simt(const DecodeArgs& a, int num_sms, cudaStream_t st);

// ------------------------------------------------------------------ linear
struct LinearLayout {
  size_t dz;         // [M][ld_dz] the pre-activation's gradient, dims->dtype
  size_t db_part;    // [kDbSplit][N] fp32
  size_t part;       // fp32 partial sums of products with a divided K
  size_t x_copy, w_copy;   // bf16 [M][ld_copy], [N][ld_copy] for rows that are not whole vectors
  int64_t ld_dz, ld_copy;
  size_t total;
};
constexpr int kDbSplit = 256;
constexpr int kMaxWidth = 65535 * 64;   // N and K of a linear layer
LinearLayout linear_layout(const moe_linear_dims& d);

// C [M, N] = A B^T, A (m, k) at a[m * am + k * ak], B (n, k) at b[n * bn + k * bk], one of the two
// strides of each being 1; C (m, n) at c[m * ldc + n].
struct GemmArgs {
  const void *a, *b;
  int64_t am, ak, bn, bk;
  int64_t M;
  int N;
  int64_t K;
  // epilogue: z = acc + bias[n]; z_out [M][ld_z]; c = act(z) + res
  const void* bias;
  const void* res;
  int64_t ld_res;
  int act;
  void* z_out;
  int64_t ld_z;      // N rounded up to a multiple of 8
  void* c;
  int64_t ldc;
  int dtype;
};
// The FMA products (fp32): shares of a divided K, and of all tiles; fp32 partial sums [tile][share][128][64].
constexpr int kMaxSplit = 32, kMaxShares = 1024;
size_t gemm_simt_part_bytes(int64_t M, int64_t N, int64_t K);   // enough for smaller ones too
cudaError_t launch_gemm_simt(const GemmArgs& g, float* part, int num_sms, cudaStream_t st);
// The bf16 products on CTA pairs. LINEAR_FWD: A and B K-major; DX: B MN-major; DW: both. Base
// pointers 16-byte aligned, row strides multiples of 8 elements.
enum LinearKind { LINEAR_FWD = 0, LINEAR_DX, LINEAR_DW };
constexpr int kMaxPairs = 80;     // clusters of two CTAs
constexpr int kMinRun = 4;        // K blocks of a pair's run when there are fewer tiles than pairs (2, 8: the same)
size_t linear_pair_part_bytes();
int launch_linear_pair(int kind, const GemmArgs& a, uint8_t* ws, size_t part, int num_sms, cudaStream_t st);
// The forward product for at most kStreamRows rows, as a stream of the weights (N = 7680, K = 2048, 64
// rows: 11.1 us, 12.4 on pairs; N = 32768, K = 1024, 128 rows: 23.4, 20.3), for up to kStreamRowsLong if
// K is kStreamLong or more (N = K = 7680, 128 rows: 29.3, 35.4; N = 2048, K = 2816: 11.8, 12.1).
constexpr int kStreamRows = 64, kStreamRowsLong = 128, kStreamLong = 2800;
int launch_linear_stream(const GemmArgs& a, uint8_t* ws, int num_sms, cudaStream_t st);
// dz = dy * act'(z) (dz may be NULL: sums only) and db (may be NULL); z and dz have ld_dz = N rounded
// up to a multiple of 8 elements between rows
cudaError_t launch_linear_dz(const void* dy, int64_t ld_dy, const void* z, int act, int64_t M, int N,
                             int dtype, void* dz, int64_t ld_dz, float* db_part, void* db, cudaStream_t st);

// ------------------------------------------------------------------ verify
struct VerifyArgs {
  const int32_t *tokens, *len;
  const void *q, *p;
  const float *u_accept, *u_sample;
  int32_t *out, *accepted;
  int64_t B, ld_q, ld_p;
  int n, V, dtype;
};
cudaError_t launch_verify(const VerifyArgs& v, int num_sms, cudaStream_t st);

// ------------------------------------------------------------------ layer norm
constexpr int kNormMaxN = 32768;   // a row in the registers of 1024 threads
constexpr int kNormParts = 512;    // most partial sums of a column
struct NormArgs {
  const void *x, *res, *w, *b;
  void *sum, *y;
  float* stats;      // [M][2]: mean, rstd
  int64_t M, ld_x, ld_res, ld_sum, ld_y;
  int N;
  float eps, inv_n;
};
struct NormBwdArgs {
  const void *x, *res, *dy, *d_sum, *w;
  const float* stats;
  void *dx, *dw, *db;
  float* part;       // [parts][2][N, rounded up to 4] partial sums of the columns
  int64_t M, ld_x, ld_res, ld_dy, ld_ds, ld_dx;
  int N;
  float inv_n;
};
cudaError_t launch_norm_fwd(const NormArgs& a, int dtype, int w_dtype, int num_sms, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, int w_dtype, int num_sms, cudaStream_t st);

// ------------------------------------------------------------------ log probabilities
constexpr int kMaxTop = 32;   // alternatives
struct LogprobArgs {
  const void* x;
  const int32_t* tokens;
  float *logprob, *stats, *entropy;   // stats [M][2]: maximum, ln sum e^(x - maximum); [M][4] if kept: the entropy too
  int32_t* top_idx;
  float* top_logprob;
  int64_t M, ld;
  int V, n_top;
  bool keep_entropy;
};
struct LogprobBwdArgs {
  const void* x;
  const int32_t* tokens;
  const float *stats, *entropy, *d_logprob, *d_entropy;
  void* dx;
  int64_t M, ld, ld_dx;
  int V;
  bool keep_entropy;   // entropy: not read, it is in stats
};
cudaError_t launch_logprob(const LogprobArgs& a, int dtype, int num_sms, cudaStream_t st);
cudaError_t launch_logprob_bwd(const LogprobBwdArgs& a, int dtype, int num_sms, cudaStream_t st);

// ------------------------------------------------------------------ clipping
constexpr int kClipFew = 16, kClipMany = 512;   // tensors of a launch (its parameters: 34 bytes for each)
constexpr int kClipParts = 1024;                // most partial sums of a launch
constexpr size_t kClipCounter = 64;             // in a workspace's header, where no other operator counts
constexpr int64_t kClipMaxTotal = 1ll << 44;    // elements of all tensors
struct alignas(16) ClipPart {   // a block's sum of squares: hi + lo + far
  float hi, lo;
  double far;
};
struct ClipArgs {
  const moe_grad* grads;   // host
  int64_t count;
  float max_norm;
  float *norm, *scale;     // device, or NULL
  ClipPart* part;
  uint32_t* counter;       // 0 between calls
};
cudaError_t launch_clip(const ClipArgs& a, int num_sms, cudaStream_t st);

}  // namespace moe
