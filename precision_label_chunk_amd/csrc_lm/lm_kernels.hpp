// Internal interface between the C entries of the language-model operators (lm_capi.cpp) and their
// kernels. Status codes, weight formats and the device's properties are those of the head's step.
#pragma once
#include "../csrc/step_kernels.hpp"

namespace elmo {

// element types of the language-model operators' tensors
constexpr int T_F32_ = 0, T_BF16_ = 1, T_F16_ = 2;

// log probabilities of given tokens with entropy and top alternatives, and their gradient
struct LogprobLayout { int segs; size_t part, keys, total; };
LogprobLayout logprobs_layout(int64_t N, int64_t V, int k);
int run_logprobs(const void* Z, int ztype, int64_t N, int64_t V, int64_t ldz, const int32_t* ids, int M, int k,
                 float* logp, float* entropy, float* row_max, float* log_sum, int32_t* top_idx, float* top_logp,
                 const LogprobLayout& s, void* workspace, hipStream_t st);
int run_logprobs_grad(const void* Z, int ztype, int64_t N, int64_t V, int64_t ldz, const int32_t* ids, int M,
                      const float* row_max, const float* log_sum, const float* entropy, const float* dlogp,
                      const float* dentropy, const float* dlse, void* dZ, int64_t ldd, hipStream_t st);

// products of a few BF16 feature rows with 4-bit weights (MXFP4 rows, or integer codes with group scales)
constexpr int W_INT4_ = 3;
int run_w4_matvec(const void* W, int wdtype, int64_t L, int D, int group, const uint16_t* scales, const uint8_t* zeros,
                  const void* X, int N, int64_t ldx, void* Y, int ytype, int64_t ldy, hipStream_t st);

// activations kept in 8 bits (E4M3 with an E8M0 scale per 32 features) and their use in the backward
struct WgradLayout { int big, tiles_o, tiles_d, segs; int64_t per; size_t total; };
int run_ckpt8_save(const void* x, int type, int64_t T, int D, int64_t ldx, int act, uint8_t* codes, uint8_t* scales,
                   void* y, int64_t ldy, hipStream_t st);
int run_ckpt8_load(const uint8_t* codes, const uint8_t* scales, int64_t T, int D, void* x, int type, int64_t ldx,
                   hipStream_t st);
int run_ckpt8_act_grad(const void* dy, int type, int64_t T, int D, int64_t lddy, int act, const uint8_t* codes,
                       const uint8_t* scales, void* dx, int64_t lddx, hipStream_t st);
WgradLayout wgrad_layout(int64_t T, int O, int D);
int run_ckpt8_wgrad(const void* dY, int64_t ldy, const uint8_t* codes, const uint8_t* scales, int64_t T, int O, int D,
                    float* dW, int accumulate, const WgradLayout& s, void* workspace, hipStream_t st);

}  // namespace elmo
