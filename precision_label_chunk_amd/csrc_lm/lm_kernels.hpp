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

// threads of one launch: a grid of 2^32 or more is cut short without an error
constexpr int64_t MAX_THREADS = int64_t(1) << 31;

// log probabilities of given labels from features and weights, and the gradients of both
// (shapes: the numbers of their tile shapes)
struct LinearLayout { int shape; int64_t parts; size_t part, given, total; };
LinearLayout linear_layout(int64_t N, int64_t V, int D, int M);
int run_linear_logprobs(const void* X, const void* W, int type, int64_t N, int64_t V, int D, int64_t ldx, int64_t ldw,
                        const int32_t* ids, int M, float* logp, float* row_max, float* log_sum, const LinearLayout& s,
                        void* workspace, hipStream_t st);
struct LinearGradLayout {
  int64_t piece, x_per, w_per;                             // labels per piece; labels / tokens per run
  int x_slots, w_slots;                                    // runs
  int logits, w_shape, x_shape;                            // tile shapes of the logits, of dW and of dX
  int planes, w_planes, x_planes;                          // 16-bit numbers whose sum holds an element of G; those that dW and dX take
  bool sum_x;                                              // dX is the sum of several runs, pieces or planes
  size_t most, inv, coef, up, G, xpart, wpart, total;
};
struct LinearGradCall {
  const void *X, *W; int type; int64_t N, V; int D; int64_t ldx, ldw;
  const int32_t* ids; int M;
  const float *row_max, *log_sum, *dlogp, *dlse;
  void* dX; int dx_type; int64_t lddx;
  void* dW; int dw_type; int64_t lddw; int accumulate;
};
enum ResultKind { NO_RESULT, RESULT_16, RESULT_32 };       // by its element type's bits
LinearGradLayout linear_grad_layout(int64_t N, int64_t V, int D, int M, int64_t chunk, ResultKind dx, ResultKind dw);
int run_zero_rows(void* out, int type, int64_t rows, int D, int64_t ld, hipStream_t st);
int run_linear_logprobs_grad(const LinearGradCall& c, const LinearGradLayout& s, void* workspace, hipStream_t st);

// rows in 8-bit integers with a scale each, and products of such rows
struct I8Layout { int shape, slots, per; int64_t L4; size_t total; };
int run_i8_quantize(const void* x, int type, int64_t N, int D, int64_t ldx, int8_t* codes, float* scales, hipStream_t st);
I8Layout i8_layout(int64_t N, int64_t L, int D);
int run_i8_matmul(const int8_t* X, const float* sx, const int8_t* W, const float* sw, int64_t N, int64_t L, int D, void* Y,
                  int ytype, int64_t ldy, const I8Layout& s, void* workspace, hipStream_t st);

// dropout from a counter-based generator (r: residual or NULL; step_at: added to step, or NULL)
int run_dropout(const void* x, int type, int64_t T, int64_t D, int64_t ldx, const void* r, int64_t ldr, uint32_t limit,
                uint64_t seed, uint64_t step, const uint64_t* step_at, uint64_t first, void* y, int64_t ldy, hipStream_t st);

}  // namespace elmo
