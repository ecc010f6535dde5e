// C ABI of the elmo_xmc library (declared in include/elmo_xmc.h): argument validation on the host,
// then the internal launchers. Nothing here allocates device memory or synchronises, except
// elmo_xmc_step_flags, which copies one word back by design.
#include "../../include/elmo_xmc.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>

#include "step_kernels.hpp"

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// the weight format, and the feature sizes it supports (MXFP4 rows must be 8-byte aligned)
int check_format(int wdtype, int D) {
  if (wdtype != ELMO_W_BF16 && wdtype != ELMO_W_E4M3 && wdtype != ELMO_W_MXFP4) return ELMO_EDTYPE;
  if (wdtype == ELMO_W_MXFP4 && D % 256 != 0) return ELMO_ESHAPE;
  return ELMO_OK;
}

int check_shapes(int B, int D, int64_t L) {
  if (B < 1 || B > ELMO_MAX_B) return ELMO_ESHAPE;
  if (D < 64 || D > ELMO_MAX_D || D % 64 != 0) return ELMO_ESHAPE;
  if (L < 1 || L >= (int64_t(1) << 31)) return ELMO_ESHAPE;
  return ELMO_OK;
}

// element type and alignment of the language-model operators' tensors
bool known_type(int t) { return t == ELMO_T_F32 || t == ELMO_T_BF16 || t == ELMO_T_F16; }
bool aligned_to(const void* p, size_t n) { return (uintptr_t)p % n == 0; }
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

// which kernels a step runs: the faster for its shape (the single pass where it is built, B <= 32
// and D = 256, 512 or 768), or the one the caller names
enum { PATH_AUTO = 0, PATH_TWO_KERNEL = 1, PATH_SINGLE = 2 };

int step_entry(void* W, int wdtype, int64_t L, int D, const void* X, int B, const int32_t* row_ptr,
               const int32_t* ids, int64_t nnz, float lr, uint64_t seed, uint64_t step, int64_t chunk, float* dX,
               float* loss_sum, uint16_t* g_out, void* workspace, size_t workspace_bytes, void* stream,
               int path) {
  int rc = check_format(wdtype, D);
  if (rc != ELMO_OK) return rc;
  if ((rc = check_shapes(B, D, L)) != ELMO_OK) return rc;
  if (chunk < 1 || nnz < 0 || !std::isfinite(lr)) return ELMO_EINVAL;
  if (!W || !X || !row_ptr || !dX || (nnz > 0 && !ids)) return ELMO_EINVAL;
  if (!aligned16(W) || !aligned16(X) || !aligned16(dX)) return ELMO_EINVAL;
  const bool fits = elmo::single_pass_shape(elmo::padded_batch(B), D);
  if (path == PATH_SINGLE && !fits) return ELMO_EUNSUPPORTED;
  const bool single = path == PATH_SINGLE || (path == PATH_AUTO && fits);
  if (!workspace || !aligned16(workspace)) return ELMO_EWORKSPACE;
  const elmo::StepLayout s = elmo::step_layout(B, D, L, chunk, wdtype, nnz);
  if (workspace_bytes < s.total) return ELMO_EWORKSPACE;
  elmo::StepArgs a{};
  a.W = W; a.wdtype = wdtype; a.L = L; a.D = D; a.X = X; a.B = B;
  a.row_ptr = row_ptr; a.ids = ids; a.nnz = nnz; a.lr = lr; a.seed = seed; a.step = step;
  a.dX = dX; a.loss = loss_sum; a.l0 = 0; a.l1 = L; a.Z = nullptr; a.single = single;
  a.Gout = g_out;                        // (single pass only: its diagnostic gradient copy)
  return elmo::run_step(a, s, workspace, (hipStream_t)stream);
}

}  // namespace

extern "C" {

int elmo_abi_version(void) { return 1; }

const char* elmo_status_str(int status) {
  switch (status) {
    case ELMO_OK: return "ok";
    case ELMO_EINVAL: return "invalid argument";
    case ELMO_ESHAPE: return "unsupported shape";
    case ELMO_EDTYPE: return "unknown weight format";
    case ELMO_EWORKSPACE: return "workspace missing or too small";
    case ELMO_EHIP: return "HIP runtime error";
    case ELMO_EUNSUPPORTED: return "not supported by this library";
    case ELMO_ESCRATCH: return "step needs more scratch than the allocation-free entry point's static buffer holds";
    default: return "unknown status";
  }
}

size_t elmo_xmc_step_workspace_bytes(int B, int D, int64_t L, int64_t chunk, int wdtype, int64_t max_nnz) {
  if (check_shapes(B, D, L) != ELMO_OK || chunk < 1 || max_nnz < 0) return 0;
  if (check_format(wdtype, D) != ELMO_OK) return 0;
  return elmo::step_layout(B, D, L, chunk, wdtype, max_nnz).total;
}

int elmo_xmc_step(void* W, int wdtype, int64_t L, int D, const void* X, int B, const int32_t* row_ptr,
                  const int32_t* ids, int64_t nnz, float lr, uint64_t seed, uint64_t step, int64_t chunk,
                  float* dX, float* loss_sum, void* workspace, size_t workspace_bytes, void* stream) {
  return step_entry(W, wdtype, L, D, X, B, row_ptr, ids, nnz, lr, seed, step, chunk, dX, loss_sum, nullptr,
                    workspace, workspace_bytes, stream, PATH_AUTO);
}

int elmo_xmc_step_two_kernel(void* W, int wdtype, int64_t L, int D, const void* X, int B, const int32_t* row_ptr,
                             const int32_t* ids, int64_t nnz, float lr, uint64_t seed, uint64_t step, int64_t chunk,
                             float* dX, float* loss_sum, void* workspace, size_t workspace_bytes, void* stream) {
  return step_entry(W, wdtype, L, D, X, B, row_ptr, ids, nnz, lr, seed, step, chunk, dX, loss_sum, nullptr,
                    workspace, workspace_bytes, stream, PATH_TWO_KERNEL);
}

int elmo_xmc_step_single_pass(void* W, int wdtype, int64_t L, int D, const void* X, int B, const int32_t* row_ptr,
                              const int32_t* ids, int64_t nnz, float lr, uint64_t seed, uint64_t step,
                              int64_t chunk, float* dX, float* loss_sum, uint16_t* g_out, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (g_out && ((uintptr_t)g_out & 1u)) return ELMO_EINVAL;
  return step_entry(W, wdtype, L, D, X, B, row_ptr, ids, nnz, lr, seed, step, chunk, dX, loss_sum, g_out,
                    workspace, workspace_bytes, stream, PATH_SINGLE);
}

int elmo_xmc_step_noalloc(void* W, int wdtype, int64_t L, int D, const void* X, int B, const int32_t* row_ptr,
                          const int32_t* ids, int64_t nnz, float lr, uint64_t seed, uint64_t step, int64_t chunk,
                          float* dX, float* loss_sum, void* stream) {
  int rc = check_format(wdtype, D);
  if (rc != ELMO_OK) return rc;
  if ((rc = check_shapes(B, D, L)) != ELMO_OK) return rc;
  if (chunk < 1 || nnz < 0 || !std::isfinite(lr)) return ELMO_EINVAL;
  if (!W || !X || !row_ptr || !dX || (nnz > 0 && !ids)) return ELMO_EINVAL;
  if (!aligned16(W) || !aligned16(X) || !aligned16(dX)) return ELMO_EINVAL;
  const elmo::StepLayout s = elmo::step_layout(B, D, L, chunk, wdtype, nnz);
  if (s.total > (size_t)ELMO_NOALLOC_SCRATCH_BYTES) return ELMO_ESCRATCH;
  void* ws = nullptr;
  if ((rc = elmo::noalloc_scratch(&ws)) != ELMO_OK) return rc;
  elmo::StepArgs a{};
  a.W = W; a.wdtype = wdtype; a.L = L; a.D = D; a.X = X; a.B = B;
  a.row_ptr = row_ptr; a.ids = ids; a.nnz = nnz; a.lr = lr; a.seed = seed; a.step = step;
  a.dX = dX; a.loss = loss_sum; a.l0 = 0; a.l1 = L; a.Z = nullptr;
  return elmo::run_step(a, s, ws, (hipStream_t)stream);
}

int elmo_xmc_step_flags(const void* workspace, uint32_t* flags, void* stream) {
  if (!workspace || !flags) return ELMO_EINVAL;
  if (hipMemcpyAsync(flags, workspace, sizeof(uint32_t), hipMemcpyDeviceToHost, (hipStream_t)stream) != hipSuccess)
    return ELMO_EHIP;
  if (hipStreamSynchronize((hipStream_t)stream) != hipSuccess) return ELMO_EHIP;
  return ELMO_OK;
}

int elmo_xmc_forward(const void* W, int wdtype, int64_t L, int D, const void* X, int B, const int32_t* row_ptr,
                     const int32_t* ids, int64_t nnz, int64_t l0, int64_t l1, float* Z, uint16_t* G,
                     void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_format(wdtype, D);
  if (rc != ELMO_OK) return rc;
  if ((rc = check_shapes(B, D, L)) != ELMO_OK) return rc;
  if (l0 < 0 || l1 > L || l1 <= l0) return ELMO_ESHAPE;
  if (nnz < 0 || (nnz > 0 && (!ids || !row_ptr))) return ELMO_EINVAL;
  if (!W || !X || (!Z && !G) || !aligned16(W) || !aligned16(X)) return ELMO_EINVAL;
  if (!workspace || !aligned16(workspace)) return ELMO_EWORKSPACE;
  const elmo::StepLayout s = elmo::step_layout(B, D, L, l1 - l0, wdtype, nnz);
  if (workspace_bytes < s.total) return ELMO_EWORKSPACE;
  elmo::StepArgs a{};
  a.W = const_cast<void*>(W); a.wdtype = wdtype; a.L = L; a.D = D; a.X = X; a.B = B;
  a.row_ptr = row_ptr; a.ids = ids; a.nnz = nnz;
  a.l0 = l0 - l0 % elmo::TJ1; a.l1 = l1;
  a.Z = Z; a.Gout = G; a.zpitch = l1 - l0; a.zoff = l0;
  return elmo::run_step(a, s, workspace, (hipStream_t)stream);
}

int elmo_xmc_logits(const void* W, int wdtype, int64_t L, int D, int64_t l0, int64_t l1, const void* X, int B,
                    float* Z, void* workspace, size_t workspace_bytes, void* stream) {
  if (!Z) return ELMO_EINVAL;
  return elmo_xmc_forward(W, wdtype, L, D, X, B, nullptr, nullptr, 0, l0, l1, Z, nullptr, workspace,
                          workspace_bytes, stream);
}

size_t elmo_xmc_topk_workspace_bytes(int N, int D, int64_t L, int k, int wdtype) {
  if (N < 1 || D < 64 || D > ELMO_MAX_D || D % 64 != 0 || L < 1 || L >= (int64_t(1) << 31)) return 0;
  if (k < 1 || k > ELMO_MAX_TOPK || k > L) return 0;
  if (check_format(wdtype, D) != ELMO_OK) return 0;
  return elmo::topk_layout(N, D, L, k, wdtype).total;
}

int elmo_xmc_topk(const void* W, int wdtype, int64_t L, int D, const void* X, int N, int k, int32_t* out_idx,
                  float* out_score, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_format(wdtype, D);
  if (rc != ELMO_OK) return rc;
  if (N < 1 || D < 64 || D > ELMO_MAX_D || D % 64 != 0 || L < 1 || L >= (int64_t(1) << 31)) return ELMO_ESHAPE;
  if (k < 1 || k > ELMO_MAX_TOPK || k > L) return ELMO_ESHAPE;
  if (!W || !X || !out_idx || !aligned16(W) || !aligned16(X)) return ELMO_EINVAL;
  if (!workspace || !aligned16(workspace)) return ELMO_EWORKSPACE;
  const elmo::TopkLayout s = elmo::topk_layout(N, D, L, k, wdtype);
  if (workspace_bytes < s.total) return ELMO_EWORKSPACE;
  return elmo::run_topk(W, wdtype, L, D, X, N, k, out_idx, out_score, s, workspace, (hipStream_t)stream);
}

int elmo_xmc_kernel_timing(int enable) {
  elmo::kernel_timing_enable(enable);
  return ELMO_OK;
}

int elmo_xmc_kernel_timing_read(double* ms, int64_t* launches, double* labels) {
  if (!ms || !launches || !labels) return ELMO_EINVAL;
  return elmo::kernel_timing_read(ms, launches, labels);
}

int elmo_kahan_update(uint16_t* w, uint16_t* c, const float* g, int64_t n, float lr, void* stream) {
  if (n < 0) return ELMO_ESHAPE;
  if (n == 0) return ELMO_OK;
  if (!w || !c || !g || (uintptr_t)w % 2 || (uintptr_t)c % 2 || (uintptr_t)g % 4) return ELMO_EINVAL;
  return elmo::run_kahan_update(w, c, g, n, lr, (hipStream_t)stream);
}

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

int elmo_numerics_probe(int op, const void* in0, const void* in1, void* out, int64_t n, uint64_t seed,
                        uint64_t step, void* stream) {
  return elmo::run_numerics_probe(op, in0, in1, out, n, seed, step, (hipStream_t)stream);
}

}  // extern "C"
