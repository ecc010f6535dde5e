// C entries of the language-model operators (declared in include/elmo_xmc.h): argument validation on the
// host, then the internal launchers. Nothing here allocates device memory or synchronises.
#include "../../include/elmo_xmc.h"

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "lm_kernels.hpp"

namespace {

bool aligned_to(const void* p, size_t n) { return (uintptr_t)p % n == 0; }
bool aligned16(const void* p) { return aligned_to(p, 16); }

// element type and alignment of the language-model operators' tensors
bool known_type(int t) { return t == ELMO_T_F32 || t == ELMO_T_BF16 || t == ELMO_T_F16; }
size_t type_bytes(int t) { return t == ELMO_T_F32 ? 4 : 2; }

int check_rows(int ztype, int64_t N, int64_t V, int64_t ld, int M) {
  if (!known_type(ztype)) return ELMO_EDTYPE;
  if (N < 0 || N >= (int64_t(1) << 31) || V < 1 || V >= (int64_t(1) << 31) || ld < V) return ELMO_ESHAPE;
  if (M < 0 || M > ELMO_MAX_GIVEN) return ELMO_ESHAPE;
  return ELMO_OK;
}

// a [T, D] matrix with 16-byte aligned rows, and the 8-bit form of one
bool rows16(const void* p, int type, int64_t ld) { return aligned16(p) && ld * (int64_t)type_bytes(type) % 16 == 0; }
int check_ckpt8(int type, int64_t T, int D) {
  if (!known_type(type)) return ELMO_EDTYPE;
  if (T < 0 || T >= (int64_t(1) << 31) || D < 32 || D % 32 != 0 || D > (1 << 24)) return ELMO_ESHAPE;
  return ELMO_OK;
}

// features and head weights of 16-bit elements, K = D: 16-byte aligned rows, 256 of them within 2^31 bytes
constexpr int64_t MAX_LINEAR_LD = (1 << 22) - 64;
int check_linear(int type, int64_t N, int64_t V, int D, int64_t ldx, int64_t ldw, int M) {
  if (type != ELMO_T_BF16 && type != ELMO_T_F16) return ELMO_EDTYPE;
  if (N < 0 || N >= (int64_t(1) << 31) || V < 1 || V >= (int64_t(1) << 31)) return ELMO_ESHAPE;
  if (D < 32 || D % 32 != 0 || D > ELMO_MAX_LINEAR_D || M < 0 || M > ELMO_MAX_GIVEN) return ELMO_ESHAPE;
  if (ldx < D || ldw < D || ldx > MAX_LINEAR_LD || ldw > MAX_LINEAR_LD) return ELMO_ESHAPE;
  if (((N + 63) / 64) * ((V + 63) / 64) >= (int64_t(1) << 30)) return ELMO_ESHAPE;   // (tiles are counted in 31 bits)
  return ELMO_OK;
}

elmo::ResultKind result_kind(const void* p, int type) { return !p ? elmo::NO_RESULT : type == ELMO_T_F32 ? elmo::RESULT_32 : elmo::RESULT_16; }
// whether a result that is needed as the workspace's query says (0: not, 2 + its type, else in any type) may be
// of a kind (one that is not needed: the first)
bool may_be(int need, elmo::ResultKind kind) {
  if (need == 0 || need == 2 + ELMO_T_BF16 || need == 2 + ELMO_T_F16) return kind == elmo::RESULT_16;
  return need != 2 + ELMO_T_F32 || kind == elmo::RESULT_32;
}

int check_i8(int64_t N, int64_t L, int D) {
  if (N < 0 || N >= (int64_t(1) << 31) || L < 1 || L >= (int64_t(1) << 31)) return ELMO_ESHAPE;
  if (D < 64 || D % 64 != 0 || D > ELMO_MAX_I8_D) return ELMO_ESHAPE;
  if (((N + 63) / 64) * ((L + 63) / 64) >= (int64_t(1) << 30)) return ELMO_ESHAPE;
  return ELMO_OK;
}

}  // namespace

extern "C" {

size_t elmo_logprobs_workspace_bytes(int64_t N, int64_t V, int k) {
  if (check_rows(ELMO_T_F32, N, V, V, 0) != ELMO_OK || N < 1 || k < 0 || k > ELMO_MAX_TOPK || k > V) return 0;
  return elmo::logprobs_layout(N, V, k).total;
}

int elmo_logprobs(const void* Z, int ztype, int64_t N, int64_t V, int64_t ldz, const int32_t* ids, int M, int k,
                  float* logp, float* entropy, float* row_max, float* log_sum, int32_t* top_idx, float* top_logp,
                  void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_rows(ztype, N, V, ldz, M);
  if (rc != ELMO_OK) return rc;
  if (k < 0 || k > ELMO_MAX_TOPK || k > V) return ELMO_ESHAPE;
  if (N == 0) return ELMO_OK;
  if (!Z || !entropy || !row_max || !log_sum || (M > 0 && (!ids || !logp)) || (k > 0 && (!top_idx || !top_logp)))
    return ELMO_EINVAL;
  if (!aligned_to(Z, type_bytes(ztype))) return ELMO_EINVAL;
  for (const void* p : {(const void*)ids, (const void*)logp, (const void*)entropy, (const void*)row_max,
                        (const void*)log_sum, (const void*)top_idx, (const void*)top_logp})
    if (!aligned_to(p, 4)) return ELMO_EINVAL;
  if (!workspace || !aligned16(workspace)) return ELMO_EWORKSPACE;
  const elmo::LogprobLayout s = elmo::logprobs_layout(N, V, k);
  if (workspace_bytes < s.total) return ELMO_EWORKSPACE;
  return elmo::run_logprobs(Z, ztype, N, V, ldz, ids, M, k, logp, entropy, row_max, log_sum, top_idx, top_logp, s,
                            workspace, (hipStream_t)stream);
}

int elmo_logprobs_backward(const void* Z, int ztype, int64_t N, int64_t V, int64_t ldz, const int32_t* ids, int M,
                           const float* row_max, const float* log_sum, const float* entropy, const float* dlogp,
                           const float* dentropy, const float* dlse, void* dZ, int64_t ldd, void* stream) {
  const int rc = check_rows(ztype, N, V, ldz, M);
  if (rc != ELMO_OK) return rc;
  if (ldd < V || (dZ == Z && ldd != ldz)) return ELMO_ESHAPE;
  if (N == 0) return ELMO_OK;
  if (!Z || !dZ || !row_max || !log_sum || !entropy || (M > 0 && (!ids || !dlogp))) return ELMO_EINVAL;
  if (!aligned_to(Z, type_bytes(ztype)) || !aligned_to(dZ, type_bytes(ztype))) return ELMO_EINVAL;
  for (const void* p : {(const void*)ids, (const void*)row_max, (const void*)log_sum, (const void*)entropy,
                        (const void*)dlogp, (const void*)dentropy, (const void*)dlse})
    if (!aligned_to(p, 4)) return ELMO_EINVAL;
  return elmo::run_logprobs_grad(Z, ztype, N, V, ldz, ids, M, row_max, log_sum, entropy, dlogp, dentropy, dlse, dZ,
                                 ldd, (hipStream_t)stream);
}

int elmo_w4_matvec(const void* W, int wdtype, int64_t L, int D, int group, const uint16_t* scales,
                   const uint8_t* zeros, const void* X, int N, int64_t ldx, void* Y, int ytype, int64_t ldy,
                   void* stream) {
  if (wdtype != ELMO_W_MXFP4 && wdtype != ELMO_W_INT4) return ELMO_EDTYPE;
  if (!known_type(ytype)) return ELMO_EDTYPE;
  if (N < 0 || N > ELMO_MAX_MATVEC_ROWS || L < 1 || L >= (int64_t(1) << 31) || D < 1 || D > ELMO_MAX_MATVEC_D)
    return ELMO_ESHAPE;
  if (ldx < D || ldx % 8 != 0 || ldy < L) return ELMO_ESHAPE;
  if (wdtype == ELMO_W_MXFP4 && (group != 32 || D % 256 != 0)) return ELMO_ESHAPE;
  if (wdtype == ELMO_W_INT4 && ((group != 32 && group != 64 && group != 128) || D % group != 0)) return ELMO_ESHAPE;
  if (N == 0) return ELMO_OK;
  if (!W || !X || !Y || !aligned16(X) || !aligned_to(Y, type_bytes(ytype))) return ELMO_EINVAL;
  if (wdtype == ELMO_W_MXFP4 && (scales || zeros || !aligned_to(W, 8))) return ELMO_EINVAL;
  if (wdtype == ELMO_W_INT4 && (!scales || !aligned_to(scales, 2) || !aligned16(W))) return ELMO_EINVAL;
  return elmo::run_w4_matvec(W, wdtype, L, D, group, scales, zeros, X, N, ldx, Y, ytype, ldy, (hipStream_t)stream);
}

int elmo_ckpt8_save(const void* x, int type, int64_t T, int D, int64_t ldx, int act, uint8_t* codes, uint8_t* scales,
                    void* y, int64_t ldy, void* stream) {
  const int rc = check_ckpt8(type, T, D);
  if (rc != ELMO_OK) return rc;
  if (act < ELMO_ACT_NONE || act > ELMO_ACT_GELU) return ELMO_EINVAL;
  if (ldx < D || (y && ldy < D)) return ELMO_ESHAPE;
  if (T == 0) return ELMO_OK;
  if ((act == ELMO_ACT_NONE) != (y == nullptr)) return ELMO_EINVAL;
  if (!x || !codes || !scales || !rows16(x, type, ldx) || (y && !rows16(y, type, ldy)) || !aligned_to(codes, 8))
    return ELMO_EINVAL;
  return elmo::run_ckpt8_save(x, type, T, D, ldx, act, codes, scales, y, ldy, (hipStream_t)stream);
}

int elmo_ckpt8_load(const uint8_t* codes, const uint8_t* scales, int64_t T, int D, void* x, int type, int64_t ldx,
                    void* stream) {
  const int rc = check_ckpt8(type, T, D);
  if (rc != ELMO_OK) return rc;
  if (ldx < D) return ELMO_ESHAPE;
  if (T == 0) return ELMO_OK;
  if (!x || !codes || !scales || !rows16(x, type, ldx) || !aligned_to(codes, 8)) return ELMO_EINVAL;
  return elmo::run_ckpt8_load(codes, scales, T, D, x, type, ldx, (hipStream_t)stream);
}

int elmo_ckpt8_act_grad(const void* dy, int type, int64_t T, int D, int64_t lddy, int act, const uint8_t* codes,
                        const uint8_t* scales, void* dx, int64_t lddx, void* stream) {
  const int rc = check_ckpt8(type, T, D);
  if (rc != ELMO_OK) return rc;
  if (act < ELMO_ACT_RELU || act > ELMO_ACT_GELU) return ELMO_EINVAL;
  if (lddy < D || lddx < D || (dx == dy && lddx != lddy)) return ELMO_ESHAPE;
  if (T == 0) return ELMO_OK;
  if (!dy || !dx || !codes || !scales || !rows16(dy, type, lddy) || !rows16(dx, type, lddx) || !aligned_to(codes, 8))
    return ELMO_EINVAL;
  return elmo::run_ckpt8_act_grad(dy, type, T, D, lddy, act, codes, scales, dx, lddx, (hipStream_t)stream);
}

size_t elmo_ckpt8_weight_grad_workspace_bytes(int64_t T, int O, int D) {
  if (check_ckpt8(ELMO_T_BF16, T, D) != ELMO_OK || O < 8 || O % 8 != 0 || O > (1 << 23)) return 0;
  return elmo::wgrad_layout(T, O, D).total;
}

int elmo_ckpt8_weight_grad(const void* dY, int64_t ldy, const uint8_t* codes, const uint8_t* scales, int64_t T, int O,
                           int D, float* dW, int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_ckpt8(ELMO_T_BF16, T, D);
  if (rc != ELMO_OK) return rc;
  if (O < 8 || O % 8 != 0 || ldy < O || ldy > (1 << 23) || ldy % 8 != 0) return ELMO_ESHAPE;
  if (!dW || !aligned16(dW)) return ELMO_EINVAL;
  if (T > 0 && (!dY || !codes || !scales || !aligned16(dY) || !aligned_to(codes, 8))) return ELMO_EINVAL;
  if (!workspace || !aligned16(workspace)) return ELMO_EWORKSPACE;
  const elmo::WgradLayout s = elmo::wgrad_layout(T, O, D);
  if (workspace_bytes < s.total) return ELMO_EWORKSPACE;
  return elmo::run_ckpt8_wgrad(dY, ldy, codes, scales, T, O, D, dW, accumulate, s, workspace, (hipStream_t)stream);
}

size_t elmo_linear_logprobs_workspace_bytes(int64_t N, int64_t V, int D, int M) {
  if (N < 1 || check_linear(ELMO_T_BF16, N, V, D, D, D, M) != ELMO_OK) return 0;
  return elmo::linear_layout(N, V, D, M).total;
}

int elmo_linear_logprobs(const void* X, const void* W, int type, int64_t N, int64_t V, int D, int64_t ldx, int64_t ldw,
                         const int32_t* ids, int M, float* logp, float* row_max, float* log_sum, void* workspace,
                         size_t workspace_bytes, void* stream) {
  const int rc = check_linear(type, N, V, D, ldx, ldw, M);
  if (rc != ELMO_OK) return rc;
  if (N == 0) return ELMO_OK;
  if (!X || !W || !row_max || !log_sum || (M > 0 && (!ids || !logp))) return ELMO_EINVAL;
  if (!rows16(X, type, ldx) || !rows16(W, type, ldw)) return ELMO_EINVAL;
  for (const void* p : {(const void*)ids, (const void*)logp, (const void*)row_max, (const void*)log_sum})
    if (!aligned_to(p, 4)) return ELMO_EINVAL;
  if (!workspace || !aligned16(workspace)) return ELMO_EWORKSPACE;
  const elmo::LinearLayout s = elmo::linear_layout(N, V, D, M);
  if (workspace_bytes < s.total) return ELMO_EWORKSPACE;
  return elmo::run_linear_logprobs(X, W, type, N, V, D, ldx, ldw, ids, M, logp, row_max, log_sum, s, workspace,
                                   (hipStream_t)stream);
}

size_t elmo_linear_logprobs_backward_workspace_bytes(int64_t N, int64_t V, int D, int M, int64_t chunk, int need_dx,
                                                     int need_dw) {
  if (N < 1 || chunk < 0 || check_linear(ELMO_T_BF16, N, V, D, D, D, M) != ELMO_OK) return 0;
  // a type that is not told: the largest workspace of any
  size_t most = 0;
  for (const elmo::ResultKind dx : {elmo::RESULT_16, elmo::RESULT_32})
    for (const elmo::ResultKind dw : {elmo::RESULT_16, elmo::RESULT_32}) {
      if (!may_be(need_dx, dx) || !may_be(need_dw, dw)) continue;
      const size_t total = elmo::linear_grad_layout(N, V, D, M, chunk, need_dx ? dx : elmo::NO_RESULT, need_dw ? dw : elmo::NO_RESULT).total;
      most = total > most ? total : most;
    }
  return most;
}

int elmo_linear_logprobs_backward(const void* X, const void* W, int type, int64_t N, int64_t V, int D, int64_t ldx,
                                  int64_t ldw, const int32_t* ids, int M, const float* row_max, const float* log_sum,
                                  const float* dlogp, const float* dlse, void* dX, int dx_type, int64_t lddx, void* dW,
                                  int dw_type, int64_t lddw, int accumulate, int64_t chunk, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  const int rc = check_linear(type, N, V, D, ldx, ldw, M);
  if (rc != ELMO_OK) return rc;
  if ((dX && !known_type(dx_type)) || (dW && !known_type(dw_type))) return ELMO_EDTYPE;
  if (chunk < 0 || (dX && lddx < D) || (dW && lddw < D)) return ELMO_ESHAPE;
  if (!dX && !dW) return ELMO_EINVAL;
  if (N == 0 && !dW) return ELMO_OK;
  if ((dX && !rows16(dX, dx_type, lddx)) || (dW && !rows16(dW, dw_type, lddw))) return ELMO_EINVAL;
  if (N == 0) return accumulate ? ELMO_OK : elmo::run_zero_rows(dW, dw_type, V, D, lddw, (hipStream_t)stream);
  if (!X || !W || !row_max || !log_sum || (M > 0 && (!ids || !dlogp))) return ELMO_EINVAL;
  if (!rows16(X, type, ldx) || !rows16(W, type, ldw)) return ELMO_EINVAL;
  for (const void* p : {(const void*)ids, (const void*)dlogp, (const void*)row_max, (const void*)log_sum, (const void*)dlse})
    if (!aligned_to(p, 4)) return ELMO_EINVAL;
  if (!workspace || !aligned16(workspace)) return ELMO_EWORKSPACE;
  const elmo::LinearGradLayout s = elmo::linear_grad_layout(N, V, D, M, chunk, result_kind(dX, dx_type), result_kind(dW, dw_type));
  if (workspace_bytes < s.total) return ELMO_EWORKSPACE;
  elmo::LinearGradCall c{};
  c.X = X; c.W = W; c.type = type; c.N = N; c.V = V; c.D = D; c.ldx = ldx; c.ldw = ldw; c.ids = ids; c.M = M;
  c.row_max = row_max; c.log_sum = log_sum; c.dlogp = dlogp; c.dlse = dlse;
  c.dX = dX; c.dx_type = dx_type; c.lddx = lddx; c.dW = dW; c.dw_type = dw_type; c.lddw = lddw; c.accumulate = accumulate;
  return elmo::run_linear_logprobs_grad(c, s, workspace, (hipStream_t)stream);
}

int elmo_i8_quantize(const void* x, int type, int64_t N, int D, int64_t ldx, int8_t* codes, float* scales, void* stream) {
  if (!known_type(type)) return ELMO_EDTYPE;
  const int rc = check_i8(N, 1, D);
  if (rc != ELMO_OK) return rc;
  if (ldx < D) return ELMO_ESHAPE;
  if (N == 0) return ELMO_OK;
  if (!x || !codes || !scales || !rows16(x, type, ldx) || !aligned16(codes) || !aligned_to(scales, 4)) return ELMO_EINVAL;
  return elmo::run_i8_quantize(x, type, N, D, ldx, codes, scales, (hipStream_t)stream);
}

size_t elmo_i8_matmul_workspace_bytes(int64_t N, int64_t L, int D) {
  if (N < 1 || check_i8(N, L, D) != ELMO_OK) return 0;
  return elmo::i8_layout(N, L, D).total;
}

int elmo_i8_matmul(const int8_t* X, const float* x_scales, const int8_t* W, const float* w_scales, int64_t N, int64_t L,
                   int D, void* Y, int ytype, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  if (!known_type(ytype)) return ELMO_EDTYPE;
  const int rc = check_i8(N, L, D);
  if (rc != ELMO_OK) return rc;
  if (ldy < L) return ELMO_ESHAPE;
  if (N == 0) return ELMO_OK;
  if (!X || !W || !x_scales || !w_scales || !Y || !aligned16(X) || !aligned16(W) || !aligned_to(x_scales, 4) ||
      !aligned_to(w_scales, 4) || !aligned_to(Y, type_bytes(ytype)))
    return ELMO_EINVAL;
  const elmo::I8Layout s = elmo::i8_layout(N, L, D);
  if (s.total > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < s.total)) return ELMO_EWORKSPACE;
  return elmo::run_i8_matmul(X, x_scales, W, w_scales, N, L, D, Y, ytype, ldy, s, workspace, (hipStream_t)stream);
}

int elmo_dropout(const void* x, int type, int64_t T, int64_t D, int64_t ldx, const void* residual, int64_t ldr, double p,
                 uint64_t seed, uint64_t step, const uint64_t* step_at, uint64_t first, void* y, int64_t ldy, void* stream) {
  if (!known_type(type)) return ELMO_EDTYPE;
  if (T < 0 || T >= (int64_t(1) << 31) || D < 1 || D >= (int64_t(1) << 31)) return ELMO_ESHAPE;
  if (ldx < D || ldy < D || (residual && ldr < D) || (y == x && ldy != ldx) || (residual && y == residual && ldy != ldr))
    return ELMO_ESHAPE;
  // (indices end below 2^64 - 7: blocks of 8 are counted by rounding up)
  if (!(p >= 0.0 && p <= 1.0) || first > UINT64_MAX - 7 - (uint64_t)(T * D)) return ELMO_EINVAL;
  if (T == 0) return ELMO_OK;
  const size_t e = type_bytes(type);
  if (!x || !y || !aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(residual, e) || !aligned_to(step_at, 8)) return ELMO_EINVAL;
  return elmo::run_dropout(x, type, T, D, ldx, residual, ldr, (uint32_t)(p * 65536.0 + 0.5), seed, step, step_at, first, y, ldy,
                           (hipStream_t)stream);
}

}  // extern "C"
