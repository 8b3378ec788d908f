// C ABI of the few-token operators: argument validation, workspace layouts and launches.
#include <string.h>

#include "ops.h"

namespace moe {

DecodeLayout decode_layout(const moe_dims& d) {
  DecodeLayout L;
  size_t o = kOpHeader;
  auto take = [&](size_t bytes) {
    const size_t r = o;
    o = round256(o + bytes);
    return r;
  };
  const size_t T = (size_t)d.T, E = (size_t)d.E;
  const bool tc = d.dtype == MOE_BF16;
  const size_t nt = tc ? decode_token_columns(d.T) : 0;
  L.score_part = take(4 * T * kMaxStreamCtas * E);
  L.part = take(tc ? 4 * (size_t)(kDecodeRuns + 1) * kMaxStreamCtas * nt * 128 : 0);
  const size_t rows = tc ? 2 * nt : 4 * T;   // bytes of a column of hidden rows
  L.h = take(rows * (size_t)decode_slots(d) * d.f);
  L.hs = take(rows * (size_t)d.S * d.f_s);
  L.total = o;
  return L;
}

LinearLayout linear_layout(const moe_linear_dims& d) {
  LinearLayout L;
  L.ld_dz = (d.N + 7) & ~7ll;
  L.dz = kOpHeader;
  L.db_part = L.dz + round256((size_t)d.M * L.ld_dz * elt_bytes(d.dtype));
  L.part = L.db_part + round256(4 * (size_t)kDbSplit * d.N);
  if (d.dtype == MOE_BF16) {
    L.ld_copy = (d.K + 7) & ~7ll;
    L.x_copy = L.part + round256(linear_pair_part_bytes());
    L.w_copy = L.x_copy + round256(2 * (size_t)d.M * L.ld_copy);   // a call's x may have any stride
    L.total = L.w_copy + (d.ld_w % 8 != 0 ? round256(2 * (size_t)d.N * L.ld_copy) : 0);
  } else {
    size_t part = 0;
    const size_t simt[3] = {gemm_simt_part_bytes(d.M, d.N, d.K), gemm_simt_part_bytes(d.M, d.K, d.N),
                            gemm_simt_part_bytes(d.N, d.K, d.M)};   // y, dx, dw
    for (size_t s : simt) part = s > part ? s : part;
    L.ld_copy = 0;
    L.x_copy = L.w_copy = L.total = L.part + part;
  }
  return L;
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int opt(const void* p) { return p == nullptr || aligned16(p) ? MOE_OK : MOE_ERR_MISALIGNED; }
int req(const void* p) { return p == nullptr ? MOE_ERR_NULL_POINTER : opt(p); }
int req_if(const void* p, bool needed) { return needed ? req(p) : opt(p); }

#define OP_TRY(x)                \
  do {                           \
    const int _s = (x);          \
    if (_s != MOE_OK) return _s; \
  } while (0)

int check_op_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (ws == nullptr) return MOE_ERR_NULL_POINTER;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return MOE_ERR_MISALIGNED;
  return ws_bytes < need ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

// A decode call's dims are the layer's, with few tokens and without the training variants.
int check_decode(const moe_dims* d) {
  if (d == nullptr) return MOE_ERR_NULL_POINTER;
  if (d->T > kDecodeMaxT || d->capacity != 0 || d->rearrange != 0) return MOE_ERR_BAD_DIMS;
  return check_layer_dims(d);
}

// Strides are checked with their defaults in place. M <= 2^30 rows 2^36 elements apart: offsets stay
// within 64 bits for any tensor that exists, and a tensor map's strides (below 2^40 bytes) hold them.
int resolve_linear(const moe_linear_dims* in, moe_linear_dims* d) {
  if (in == nullptr) return MOE_ERR_NULL_POINTER;
  *d = *in;
  if (d->dtype != MOE_F32 && d->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED_DTYPE;
  if (d->M < 0 || d->M > (1 << 30) || d->N < 1 || d->K < 1 || d->N > kMaxWidth || d->K > kMaxWidth) return MOE_ERR_BAD_DIMS;
  if (d->act < MOE_ACT_NONE || d->act > MOE_ACT_GELU_TANH) return MOE_ERR_BAD_DIMS;
  if (d->ld_x == 0) d->ld_x = d->K;
  if (d->ld_w == 0) d->ld_w = d->K;
  if (d->ld_y == 0) d->ld_y = d->N;
  if (d->ld_res == 0) d->ld_res = d->N;
  if (d->ld_x < d->K || d->ld_w < d->K || d->ld_y < d->N || d->ld_res < d->N || d->ld_x > kMaxLd || d->ld_w > kMaxLd ||
      d->ld_y > kMaxLd || d->ld_res > kMaxLd)
    return MOE_ERR_BAD_DIMS;
  return MOE_OK;
}

// x or w with a row stride that the TMA takes: bf16 rows that are not whole 16-byte vectors are copied
// to such first (300 x 700 x 1001: 10.6 us, 17.9 with single elements on the FMA pipes; 4096 x 2816 x
// 2047: 41 us, 1043).
int whole_vectors(const void** p, int64_t* ld, int64_t rows, const moe_linear_dims& d, int64_t ld_copy, uint8_t* copy,
                  cudaStream_t st) {
  if (d.dtype != MOE_BF16 || *ld % 8 == 0) return MOE_OK;
  if (launch_linear_dz(*p, *ld, nullptr, MOE_ACT_NONE, rows, d.K, d.dtype, copy, ld_copy, nullptr, nullptr, st) != cudaSuccess)
    return MOE_ERR_LAUNCH;
  *p = copy;
  *ld = ld_copy;
  return MOE_OK;
}

// One product of the layer: bf16 on the tensor cores, fp32 on the FMA pipes.
int run_gemm(int kind, const GemmArgs& g, uint8_t* ws, const LinearLayout& L, int sms, cudaStream_t st) {
  if (g.dtype == MOE_BF16) {
    if (kind == LINEAR_FWD && g.M <= (g.K >= kStreamLong ? kStreamRowsLong : kStreamRows)) return launch_linear_stream(g, ws, sms, st);
    return launch_linear_pair(kind, g, ws, L.part, sms, st);
  }
  return launch_gemm_simt(g, reinterpret_cast<float*>(ws + L.part), sms, st) == cudaSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

int layer_decode(const moe_layer_params* params, const void* x, const float* logits_in, const void* residual,
                 const moe_dims* dims, int32_t* topk_idx, float* topk_w, void* y, void* ws, size_t ws_bytes, uint32_t absent,
                 cudaStream_t st) {
  OP_TRY(check_decode(dims));
  if (params == nullptr) return MOE_ERR_NULL_POINTER;
  DecodeArgs a;
  memset(&a, 0, sizeof(a));
  a.L = decode_layout(*dims);
  OP_TRY(check_op_ws(ws, ws_bytes, a.L.total));
  const bool some = dims->T > 0;
  OP_TRY(req_if(x, some));
  OP_TRY(opt(logits_in));
  OP_TRY(opt(residual));
  OP_TRY(req_if(params->w_r, some && logits_in == nullptr));
  OP_TRY(opt(params->bias));
  OP_TRY(req(params->w13));
  OP_TRY(req(params->w2));
  OP_TRY(req_if(params->ws13, dims->S > 0));
  OP_TRY(req_if(params->ws2, dims->S > 0));
  OP_TRY(opt(topk_idx));
  OP_TRY(opt(topk_w));
  OP_TRY(req_if(y, some));
  if (!some) return MOE_OK;
  int sms = 0;
  OP_TRY(check_device(&sms));
  a.x = x;
  a.residual = residual;
  a.w_r = params->w_r;
  a.bias = params->bias;
  a.logits_in = logits_in;
  a.w13 = params->w13;
  a.w2 = params->w2;
  a.ws13 = params->ws13;
  a.ws2 = params->ws2;
  a.idx_out = topk_idx;
  a.gate_out = topk_w;
  a.y = y;
  a.ws = static_cast<uint8_t*>(ws);
  a.absent = absent;
  a.dm = *dims;
  return dims->dtype == MOE_BF16 ? launch_decode_tc(a, sms, st) : launch_decode_simt(a, sms, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_op_workspace_init(void* ws, size_t ws_bytes, moe_stream_t stream) {
  OP_TRY(check_op_ws(ws, ws_bytes, kOpHeader));
  return cudaMemsetAsync(ws, 0, kOpHeader, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_decode_workspace_bytes(const moe_dims* dims) {
  return check_decode(dims) == MOE_OK ? decode_layout(*dims).total : 0;
}

int moe_layer_decode(const moe_layer_params* params, const void* x, const float* logits_in, const void* residual,
                     const moe_dims* dims, int32_t* topk_idx, float* topk_w, void* y, void* ws, size_t ws_bytes,
                     moe_stream_t stream) {
  return layer_decode(params, x, logits_in, residual, dims, topk_idx, topk_w, y, ws, ws_bytes, 0, (cudaStream_t)stream);
}

int moe_debug_decode_timeout_probe(const moe_layer_params* params, const void* x, const moe_dims* dims, void* y, void* ws,
                                   size_t ws_bytes, moe_stream_t stream) {
  return layer_decode(params, x, nullptr, nullptr, dims, nullptr, nullptr, y, ws, ws_bytes, 1, (cudaStream_t)stream);
}

size_t moe_linear_workspace_bytes(const moe_linear_dims* dims) {
  moe_linear_dims d;
  return resolve_linear(dims, &d) == MOE_OK ? linear_layout(d).total : 0;
}

int moe_linear_fwd(const void* x, const void* w, const void* bias, const void* residual, const moe_linear_dims* dims,
                   void* z, void* y, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_linear_dims d;
  OP_TRY(resolve_linear(dims, &d));
  const LinearLayout L = linear_layout(d);
  OP_TRY(check_op_ws(ws, ws_bytes, L.total));
  const bool some = d.M > 0;
  OP_TRY(req_if(x, some));
  OP_TRY(req(w));
  OP_TRY(opt(bias));
  OP_TRY(opt(residual));
  OP_TRY(opt(z));
  OP_TRY(req_if(y, some));
  if (!some) return MOE_OK;
  int sms = 0;
  OP_TRY(check_device(&sms));
  uint8_t* base = static_cast<uint8_t*>(ws);
  const cudaStream_t st = (cudaStream_t)stream;
  int64_t ld_x = d.ld_x, ld_w = d.ld_w;
  OP_TRY(whole_vectors(&x, &ld_x, d.M, d, L.ld_copy, base + L.x_copy, st));
  OP_TRY(whole_vectors(&w, &ld_w, d.N, d, L.ld_copy, base + L.w_copy, st));
  GemmArgs g = {x, w, ld_x, 1, ld_w, 1, d.M, d.N, d.K, bias, residual, d.ld_res, d.act, z, L.ld_dz, y, d.ld_y, d.dtype};
  return run_gemm(LINEAR_FWD, g, base, L, sms, st);
}

int moe_linear_bwd(const void* x, const void* w, const void* z, const void* dy, const moe_linear_dims* dims, void* dx,
                   void* dw, void* db, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_linear_dims d;
  OP_TRY(resolve_linear(dims, &d));
  const LinearLayout L = linear_layout(d);
  OP_TRY(check_op_ws(ws, ws_bytes, L.total));
  const bool some = d.M > 0;
  OP_TRY(req_if(x, some && dw != nullptr));
  OP_TRY(req_if(w, dx != nullptr));
  OP_TRY(req_if(z, some && d.act != MOE_ACT_NONE));
  OP_TRY(req_if(dy, some));
  OP_TRY(opt(dx));
  OP_TRY(opt(dw));
  OP_TRY(opt(db));
  const cudaStream_t st = (cudaStream_t)stream;
  const size_t es = elt_bytes(d.dtype);
  if (!some) {
    if (dw != nullptr && cudaMemset2DAsync(dw, d.ld_w * es, 0, d.K * es, d.N, st) != cudaSuccess) return MOE_ERR_CUDA;
    if (db != nullptr && cudaMemsetAsync(db, 0, d.N * es, st) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  uint8_t* base = static_cast<uint8_t*>(ws);
  int sms = 0;
  OP_TRY(check_device(&sms));
  const bool products = dx != nullptr || dw != nullptr;
  // without an activation dz is dy itself, unless dy's rows are not whole 16-byte vectors (bf16)
  const bool own_dz = products && (d.act != MOE_ACT_NONE || (d.dtype == MOE_BF16 && d.ld_y % 8 != 0));
  const void* dz = own_dz ? base + L.dz : dy;
  const int64_t ld_dz = own_dz ? L.ld_dz : d.ld_y;
  if (own_dz || db != nullptr) {
    if (launch_linear_dz(dy, d.ld_y, z, d.act, d.M, d.N, d.dtype, own_dz ? base + L.dz : nullptr, L.ld_dz,
                         reinterpret_cast<float*>(base + L.db_part), db, st) != cudaSuccess)
      return MOE_ERR_LAUNCH;
  }
  if (dx != nullptr) {   // dx [M, K] = dz W: contraction over N
    int64_t ld_w = d.ld_w;
    OP_TRY(whole_vectors(&w, &ld_w, d.N, d, L.ld_copy, base + L.w_copy, st));
    GemmArgs g = {dz, w, ld_dz, 1, 1, ld_w, d.M, d.K, d.N, nullptr, nullptr, 0, MOE_ACT_NONE, nullptr, 0, dx, d.ld_x, d.dtype};
    OP_TRY(run_gemm(LINEAR_DX, g, base, L, sms, st));
  }
  if (dw != nullptr) {   // dw [N, K] = dz^T x: contraction over M
    int64_t ld_x = d.ld_x;
    OP_TRY(whole_vectors(&x, &ld_x, d.M, d, L.ld_copy, base + L.x_copy, st));
    GemmArgs g = {dz, x, 1, ld_dz, 1, ld_x, d.N, d.K, d.M, nullptr, nullptr, 0, MOE_ACT_NONE, nullptr, 0, dw, d.ld_w, d.dtype};
    OP_TRY(run_gemm(LINEAR_DW, g, base, L, sms, st));
  }
  return MOE_OK;
}

int moe_verify_draft(const int32_t* draft_tokens, const int32_t* draft_len, const void* draft_probs,
                     const void* target_probs, const float* u_accept, const float* u_sample,
                     const moe_verify_dims* dims, int32_t* tokens, int32_t* accepted, moe_stream_t stream) {
  if (dims == nullptr) return MOE_ERR_NULL_POINTER;
  if (dims->dtype != MOE_F32 && dims->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED_DTYPE;
  if (dims->B < 0 || dims->B > (1 << 26) || dims->n < 0 || dims->n > 1024 || dims->V < 1 || dims->V > (1 << 22) ||
      (dims->ld_draft != 0 && dims->ld_draft < dims->V) || (dims->ld_target != 0 && dims->ld_target < dims->V) ||
      dims->ld_draft > kMaxLd || dims->ld_target > kMaxLd)
    return MOE_ERR_BAD_DIMS;
  const bool some = dims->B > 0, drafts = some && dims->n > 0;
  OP_TRY(req_if(draft_tokens, drafts));
  OP_TRY(opt(draft_len));
  OP_TRY(req_if(draft_probs, drafts));
  OP_TRY(req_if(target_probs, some));
  OP_TRY(req_if(u_accept, drafts));
  OP_TRY(req_if(u_sample, some));
  OP_TRY(req_if(tokens, some));
  OP_TRY(req_if(accepted, some));
  if (!some) return MOE_OK;
  int sms = 0;
  OP_TRY(check_device(&sms));
  VerifyArgs v = {draft_tokens, draft_len, draft_probs, target_probs, u_accept, u_sample, tokens, accepted,
                  dims->B, dims->ld_draft != 0 ? dims->ld_draft : dims->V,
                  dims->ld_target != 0 ? dims->ld_target : dims->V, dims->n, dims->V, dims->dtype};
  return launch_verify(v, sms, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // extern "C"
