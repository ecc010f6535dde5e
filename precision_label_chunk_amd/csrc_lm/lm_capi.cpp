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

}  // extern "C"
