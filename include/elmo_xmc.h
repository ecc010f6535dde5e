/*
 * elmo_xmc — MI355X (gfx950) library for the chunked, fused, low-precision training step of an
 * extreme-multilabel (XMC) linear classifier head, and its top-k scoring pass.
 *
 * Method: "ELMO: Efficiency via Low-precision and Peak Memory Optimization in Large Output Spaces"
 * (atlas.scime.ai summary, sections "Approach" and "Surprising findings"; arXiv 2510.11168,
 * abstract). The classifier weights are stored in pure BF16 or FP8 E4M3 with no FP32 master copy
 * and no tensor scaling; the weight gradient is fused into a momentum-free SGD update that writes
 * the weights back in place with stochastic rounding; the label dimension is processed in chunks
 * so that transient memory is bounded by one chunk.
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers (allocated by the caller on the current HIP device) unless noted.
 *     The library never allocates or frees device memory and keeps no per-call state.
 *   - `stream` is a hipStream_t (NULL = the default stream). All work is enqueued asynchronously on
 *     it; the call returns before the device finishes. Device-side faults surface at the caller's
 *     next synchronisation.
 *   - Arguments are validated on the host before anything is enqueued; a negative elmo_status is
 *     returned and nothing runs. After each launch the HIP error state is checked (ELMO_EHIP).
 *   - Pointers must be 16-byte aligned. Buffers must not alias each other.
 *   - No C++ exception crosses this interface. Nothing is printed.
 */
#ifndef ELMO_XMC_H
#define ELMO_XMC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ELMO_OK = 0,
  ELMO_EINVAL = -1,        /* null pointer, misalignment, bad scalar argument            */
  ELMO_ESHAPE = -2,        /* B, D, L, N, k or chunk outside the supported ranges        */
  ELMO_EDTYPE = -3,        /* unknown weight format                                      */
  ELMO_EWORKSPACE = -4,    /* workspace missing or smaller than the *_workspace_bytes   */
  ELMO_EHIP = -5,          /* a HIP runtime call or kernel launch failed                 */
  ELMO_EUNSUPPORTED = -6,  /* valid request that this library does not implement         */
  ELMO_ESCRATCH = -7       /* step too large for elmo_xmc_step_noalloc's static scratch  */
} elmo_status;

/* Weight storage formats. BF16: uint16 codes. E4M3: OCP FP8 E4M3FN codes (uint8; max 448, no
 * infinity, 0x7F/0xFF NaN) — the "E4M3" of the summary page's "Surprising findings".
 * MXFP4: OCP Microscaling FP4 (the FP4 weights that the summary page's "Limitations" leave to
 * micro-tensor scaling): each row is D/2 bytes of E2M1 codes (element 2i in the low nibble of byte
 * i, 2i+1 in the high nibble; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) followed by D/32 E8M0 scale
 * bytes (2^(c-127), 255 = NaN), scale b applying to elements 32b .. 32b+31: 17*D/32 bytes per row,
 * "L x D" below meaning L such rows. Requires D % 256 == 0. The forward scores against
 * E4M3-RNE(X); the update recomputes each block's scale from the new values t: X = floor(log2
 * max|t|) - 2 clamped to [-127, 127] (an all-zero block takes -127, a block with a NaN scale 255
 * and zero codes), then each element SR(t / 2^X) to E2M1 with the element's 16 random bits (the
 * same rule and draws as the other formats), saturating at magnitude 6. */
enum { ELMO_W_BF16 = 0, ELMO_W_E4M3 = 1, ELMO_W_MXFP4 = 2 };

/* Supported shapes: 1 <= B <= 256; 64 <= D <= 1024 with D % 64 == 0 (MXFP4: D % 256 == 0); 1 <= L < 2^31;
 * chunk >= 1 (rounded down internally to a multiple of 128 labels, at least 128, and capped so that
 * one chunk of weight rows stays below 2 GiB). */
#define ELMO_MAX_B 256
#define ELMO_MAX_D 1024
#define ELMO_MAX_TOPK 64

int elmo_abi_version(void);
const char* elmo_status_str(int status);

/*
 * One training step of the classifier head (summary page, "Approach": pure low-precision
 * classifier, stochastic rounding, no momentum, gradient computation fused with the SGD update,
 * label dimension chunked; arXiv abstract: "gradient fusion and chunking").
 *
 *   W        [L, D] row-major weight codes (BF16, E4M3 or MXFP4 rows per `wdtype`), updated IN PLACE.
 *   X        [B, D] row-major BF16 codes (encoder features). Read only.
 *   row_ptr  [B+1] int32, ids [nnz] int32: the positive labels of each sample in CSR form; set
 *            semantics (duplicates collapse, any order, empty rows allowed). Ids outside [0, L)
 *            are skipped and raise bit ELMO_FLAG_LABEL_RANGE in the workspace flags word;
 *            row_ptr must be non-decreasing with row_ptr[0] = 0 and row_ptr[B] = nnz (violations
 *            raise ELMO_FLAG_ROW_PTR). `nnz` is the host-side count.
 *   lr       SGD learning rate (cast to FP32 by the caller's value).
 *   seed, step  key the counter-based RNG of the stochastic rounding: Philox4x32-10 with key =
 *            seed, counter = (g, step); element idx = j*D + k belongs to block g = idx >> 3 at
 *            position p = idx & 7, which takes 16-bit half p & 1 of output word p >> 1. Calling
 *            with the same (seed, step) on the same inputs reproduces the same W bit for bit,
 *            whatever the chunk size.
 *   chunk    labels per chunk: bounds the transient G buffer to B_pad * chunk * 2 bytes.
 *   dX       [B, D] FP32, OVERWRITTEN with sum_j G[b, j] * W_old[j, :] (pre-update weights).
 *   loss_sum nullable; if given, receives the FP32 value of the summed BCE over all (b, j).
 *   workspace, workspace_bytes: at least elmo_xmc_step_workspace_bytes(...) bytes of device
 *            memory, used for label buckets, padded/cast copies of X, one chunk of G and the dX
 *            partial sums. Its first 4 bytes are the flags word after the step completes.
 * Per element: z = X~ . w_j (X~ = X, or E4M3-RNE(X) for E4M3 and MXFP4 weights), g =
 * BF16-RNE(sigmoid(z) - y), dX += g W_old, dW = g^T X, t = fmaf(-lr, dW, w), W = SR(t) (for MXFP4
 * per 32-element block, as described with the formats).
 * Kernels: the faster of the two implementations for the shape: the single-pass step of
 * elmo_xmc_step_single_pass where it is built (B <= 32 and D = 256, 512 or 768), else the
 * two-kernel step of elmo_xmc_step_two_kernel. Both follow the rule above with the same random
 * bits; they sum each logit in a different order (see elmo_xmc_step_single_pass).
 */
#define ELMO_FLAG_LABEL_RANGE 1u
#define ELMO_FLAG_ROW_PTR 2u
size_t elmo_xmc_step_workspace_bytes(int B, int D, int64_t L, int64_t chunk, int wdtype,
                                     int64_t max_nnz);
int elmo_xmc_step(void* W, int wdtype, int64_t L, int D, const void* X, int B,
                  const int32_t* row_ptr, const int32_t* ids, int64_t nnz, float lr, uint64_t seed,
                  uint64_t step, int64_t chunk, float* dX, float* loss_sum, void* workspace,
                  size_t workspace_bytes, void* stream);
/*
 * The step as two kernels per label chunk, for every supported shape (summary page, "Approach":
 * the label dimension chunked, the gradient fused with the SGD update): a forward kernel writes the
 * chunk's BF16 gradient G (the one chunk-sized transient), then a backward kernel computes dX and
 * dW from it and updates the weights in place, dW never leaving its registers. Arguments,
 * workspace, results and errors as elmo_xmc_step, which takes this path for B > 32 or D not in
 * {256, 512, 768}.
 */
int elmo_xmc_step_two_kernel(void* W, int wdtype, int64_t L, int D, const void* X, int B,
                             const int32_t* row_ptr, const int32_t* ids, int64_t nnz, float lr,
                             uint64_t seed, uint64_t step, int64_t chunk, float* dX, float* loss_sum,
                             void* workspace, size_t workspace_bytes, void* stream);
/*
 * The same step as elmo_xmc_step computed in a single pass over the weights (summary page,
 * "Approach": the classifier gradient fused with the SGD update; arXiv abstract: "gradient
 * fusion"): one kernel per label chunk holds each 32-label weight tile in LDS while it computes the
 * tile's logits, its gradient G (kept on chip), the tile's share of dX and the update, so the
 * weights are read once and written once and no chunk of G goes to device memory. Built for
 * B <= 32 and D = 256, 512 or 768 (every weight format): there each work-group keeps its B x D FP32
 * dX accumulator in registers for the whole chunk; other shapes return ELMO_EUNSUPPORTED and
 * enqueue nothing. Arguments, workspace (elmo_xmc_step_workspace_bytes), results and errors as
 * elmo_xmc_step; the weights follow the same rule with the same random bits. Logits are summed in
 * a different order than in elmo_xmc_step, so a gradient code can round the other way and move its
 * row's updated weights; both paths meet the same tolerances against the rule.
 *   g_out    nullable diagnostic: if given, [B, L] uint16 (2-byte aligned), receives the BF16
 *            gradient codes the step used (costs a write of 2 B L bytes); otherwise untouched.
 */
int elmo_xmc_step_single_pass(void* W, int wdtype, int64_t L, int D, const void* X, int B,
                              const int32_t* row_ptr, const int32_t* ids, int64_t nnz, float lr,
                              uint64_t seed, uint64_t step, int64_t chunk, float* dX,
                              float* loss_sum, uint16_t* g_out, void* workspace,
                              size_t workspace_bytes, void* stream);
/*
 * The same step for callers that cannot allocate device memory (code under HIP graph capture, tight
 * serving loops, harnesses that forbid allocation): arguments, results and errors as elmo_xmc_step,
 * with the workspace replaced by a static device array of ELMO_NOALLOC_SCRATCH_BYTES bytes inside
 * the library (one per GPU, held from the library's first use of that GPU until the process ends;
 * its address is looked up on the first call on each device). No device memory is allocated or
 * freed. A step whose workspace (elmo_xmc_step_workspace_bytes) exceeds that size returns
 * ELMO_ESCRATCH and enqueues nothing: at B = 256, D = 768 that allows chunks of up to about
 * 131,072 labels (3M-label E4M3 step: 97 MB); at B = 128, D = 768, chunks of 262,144 BF16 labels.
 * Every call on one GPU uses that GPU's array: calls that overlap on one GPU (other streams or
 * threads) race and give undefined results; serialise them. The flags word is not readable here.
 * It runs the two-kernel step (elmo_xmc_step_two_kernel) for every shape.
 */
#define ELMO_NOALLOC_SCRATCH_BYTES (128u << 20)
int elmo_xmc_step_noalloc(void* W, int wdtype, int64_t L, int D, const void* X, int B,
                          const int32_t* row_ptr, const int32_t* ids, int64_t nnz, float lr,
                          uint64_t seed, uint64_t step, int64_t chunk, float* dX, float* loss_sum,
                          void* stream);

/* Copies the flags word of a step's workspace to *flags (HOST pointer); synchronises `stream`. */
int elmo_xmc_step_flags(const void* workspace, uint32_t* flags, void* stream);

/*
 * Top-k scoring for precision@k (summary page, "Experimental setup": P@1, P@3, P@5).
 *   W [L, D] codes, X [N, D] BF16 codes (E4M3 and MXFP4 weights score against E4M3-RNE(X), as in
 *   training).
 *   out_idx [N, k] int32: labels ranked by (FP32 logit desc, label asc), NaN logits last.
 *   out_score [N, k] FP32 logits, nullable.  1 <= k <= min(ELMO_MAX_TOPK, L), N >= 1.
 */
size_t elmo_xmc_topk_workspace_bytes(int N, int D, int64_t L, int k, int wdtype);
int elmo_xmc_topk(const void* W, int wdtype, int64_t L, int D, const void* X, int N, int k,
                  int32_t* out_idx, float* out_score, void* workspace, size_t workspace_bytes,
                  void* stream);

/*
 * Diagnostic: FP32 logits Z [B, l1 - l0] (row-major) of labels [l0, l1) computed by the same
 * forward kernel the step uses. Workspace as for elmo_xmc_step with chunk = l1 - l0, nnz = 0.
 */
int elmo_xmc_logits(const void* W, int wdtype, int64_t L, int D, int64_t l0, int64_t l1,
                    const void* X, int B, float* Z, void* workspace, size_t workspace_bytes,
                    void* stream);

/*
 * Diagnostic: the step's forward kernel over labels [l0, l1) with the step's label handling,
 * writing the FP32 logits Z and/or the BF16 gradient codes G = BF16(sigmoid(Z) - Y) that a
 * two-kernel step with the same inputs uses (each [B, l1 - l0] row-major, nullable but not both;
 * the single-pass step reports its own codes through its g_out). Weights are not
 * touched. Labels as for elmo_xmc_step (row_ptr/ids may be NULL when nnz = 0). Workspace as for
 * elmo_xmc_step with chunk = l1 - l0 and max_nnz = nnz.
 */
int elmo_xmc_forward(const void* W, int wdtype, int64_t L, int D, const void* X, int B,
                     const int32_t* row_ptr, const int32_t* ids, int64_t nnz, int64_t l0, int64_t l1,
                     float* Z, uint16_t* G, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Measurement aid (off by default; process-wide, not thread-safe): while enabled, each launch of
 * the step's forward (index 0) and backward/update (index 1) kernels is bracketed by HIP events on
 * the launch stream. elmo_xmc_kernel_timing_read waits for the recorded events and fills, for each
 * of the two kernels (HOST arrays of 2): summed milliseconds, number of launches and labels
 * processed; the records are then cleared.
 */
int elmo_xmc_kernel_timing(int enable);
int elmo_xmc_kernel_timing_read(double* ms, int64_t* launches, double* labels);

/* Kahan-compensated BF16 update of n encoder parameters, in place (ELMO summary, Approach: the
 * encoder is trained with Kahan summation and no FP32 master weights; the pages fix neither the
 * compensation's precision nor the order of operations, this is one step of Kahan's compensated
 * summation of the increments). w[i]: the parameter, c[i]: its compensation, both BF16 codes;
 * g[i]: the binary32 gradient. Per element, in binary32 with both stores rounded to nearest-even:
 *   d = -lr g;  y = d - c;  t = bf16(w + y);  c = bf16((t - w) - y);  w = t.
 * w, c, g: DEVICE pointers to n elements each, naturally aligned (2, 2, 4 bytes; 16-byte alignment
 * of all three takes the vector path), owned by the caller; w and c must not overlap each other or
 * g. n = 0 is a no-op. Returns ELMO_ESHAPE for n < 0, ELMO_EINVAL for a null or misaligned
 * pointer, ELMO_EHIP on a launch failure; asynchronous on `stream`. */
int elmo_kahan_update(uint16_t* w, uint16_t* c, const float* g, int64_t n, float lr, void* stream);

/*
 * ---- Language-model operators -----------------------------------------------------------------
 * The softmax side of a large head and what a model in front of it trains and serves with. Same
 * conventions as above (device pointers, caller-owned workspaces, asynchronous, host validation);
 * pointers here need the alignment of their elements unless an entry says more.
 * Element types: */
enum { ELMO_T_F32 = 0, ELMO_T_BF16 = 1, ELMO_T_F16 = 2 };

/*
 * Log probabilities of given tokens under rows of logits, with the entropy of each row and its top
 * alternatives. All arithmetic in binary32.
 *
 *   Z        [N, V] logits of element type `ztype`, row n at Z + n ldz elements (ldz >= V), elements
 *            of a row adjacent; any row alignment. -inf is a masked token.
 *   ids      [N, M] int32, 0 <= M <= ELMO_MAX_GIVEN (NULL if M = 0). A negative id stands for no
 *            token: its log probability is 0 in any row. An id >= V gives NaN in any row.
 *   k        alternatives per row, 0 <= k <= min(ELMO_MAX_TOPK, V).
 *   logp     [N, M] FP32: (z[id] - row_max) - log_sum.
 *   entropy  [N] FP32: -sum_v p_v log p_v.
 *   row_max, log_sum  [N] FP32: m = max_v z_v and log sum_v e^(z_v - m), whose sum is the row's log
 *            partition; apart they keep log_sum's digits at logits of any magnitude.
 *   top_idx, top_logp [N, k] int32 and FP32: tokens by (logit desc, token asc), NaN logits last, and
 *            their log probabilities (both NULL if k = 0).
 * A row of nothing but -inf has row_max -inf, log_sum 0, entropy 0 and every token's log probability -inf. A
 * NaN or +inf logit makes log_sum, entropy and every token's log probability of its row NaN (row_max skips
 * NaN: -inf if there is nothing else). Results repeat bit for bit on one device; the order of a row's sums,
 * and with it their last bits, follows from N, V, ztype and the row's alignment to 16 bytes.
 * 1 <= V < 2^31, 0 <= N < 2^31 (N = 0: nothing is done).
 */
#define ELMO_MAX_GIVEN 64
size_t elmo_logprobs_workspace_bytes(int64_t N, int64_t V, int k);
int elmo_logprobs(const void* Z, int ztype, int64_t N, int64_t V, int64_t ldz, const int32_t* ids, int M, int k,
                  float* logp, float* entropy, float* row_max, float* log_sum, int32_t* top_idx, float* top_logp,
                  void* workspace, size_t workspace_bytes, void* stream);
/*
 * The gradient of the above with respect to the logits, from the upstream gradients dlogp [N, M]
 * (NULL if M = 0), dentropy [N] (nullable) and dlse [N] (nullable: of row_max + log_sum):
 *   dZ[n, v] = p_v (dlse - sum_j dlogp_j - dentropy (log p_v + H)) + sum_{j : ids_j = v} dlogp_j.
 * row_max, log_sum and entropy are elmo_logprobs' outputs for the same Z. A token given more than
 * once receives the sum of its gradients, a negative id none. A row of nothing but -inf has gradient 0,
 * whatever its ids; in any other row an id >= V makes the whole row NaN.
 *   dZ       [N, V] of type `ztype`, row n at dZ + n ldd. dZ = Z with ldd = ldz is allowed (in
 *            place); no other overlap is. No workspace.
 */
int elmo_logprobs_backward(const void* Z, int ztype, int64_t N, int64_t V, int64_t ldz, const int32_t* ids, int M,
                           const float* row_max, const float* log_sum, const float* entropy, const float* dlogp,
                           const float* dentropy, const float* dlse, void* dZ, int64_t ldd, void* stream);

/*
 * Products of a few feature rows with 4-bit weights with group scales, Y[n, j] = sum_k X[n, k] w[j, k]:
 * the logits of a 4-bit head, or any layer, for the rows of a decode step. The weights are read once;
 * features stay BF16 (elmo_xmc_logits casts them to E4M3 and reads D <= 1024), every product is exact
 * and sums are binary32. With integer codes the products are c x, summed over a group and joined with
 * its zero point and scale as s (sum c x - z sum x): the rounding is that of sums of c |x| and z |x|, and
 * these have to stay below 2^128 themselves.
 *   wdtype   ELMO_W_MXFP4: W holds L rows of 17 D / 32 bytes as described with the formats, D % 256 == 0,
 *            8-byte aligned; group = 32, scales = zeros = NULL.
 *            ELMO_W_INT4: W holds L rows of D/2 bytes, code c[2i] in the low nibble of byte i and
 *            c[2i + 1] in the high one, 16-byte aligned; w = (c - z) s with, per group of `group` (32,
 *            64 or 128, dividing D) features, s = scales[j, k / group] (BF16, [L, D / group]) and
 *            z = zeros[j, k / group] (uint8, [L, D / group]; NULL: 8 everywhere).
 *   X        [N, D] BF16, 1 <= N <= ELMO_MAX_MATVEC_ROWS (N = 0: nothing is done), row n at X + n ldx;
 *            16-byte aligned rows (ldx % 8 == 0).
 *   Y        [N, L] of element type `ytype` (rounded once from binary32), row n at Y + n ldy.
 * 1 <= L < 2^31; D <= ELMO_MAX_MATVEC_D. No workspace. Values out of range stay in the row and label they enter:
 * an MXFP4 scale of 255 (NaN), a NaN weight scale and a NaN feature make its results NaN. An MXFP4 weight of
 * 2^128 or more (scale codes 253 and 254 with the largest elements) is infinite. An infinite feature or
 * weight makes an MXFP4 result infinite (NaN against a zero, or against infinity of the other sign); an infinite
 * feature makes a result of integer codes NaN.
 */
enum { ELMO_W_INT4 = 3 };                 /* elmo_w4_matvec only */
#define ELMO_MAX_MATVEC_ROWS 32
#define ELMO_MAX_MATVEC_D 65536
int elmo_w4_matvec(const void* W, int wdtype, int64_t L, int D, int group, const uint16_t* scales,
                   const uint8_t* zeros, const void* X, int N, int64_t ldx, void* Y, int ytype, int64_t ldy,
                   void* stream);

/*
 * Activation checkpoints in 8 bits: what an encoder keeps between its forward and its backward pass,
 * at 33/32 of a byte per element, and the two uses of it in the backward.
 *
 * Format: codes [T, D] OCP E4M3 bytes and scales [T, D / 32] E8M0 bytes (both row-major, 8-byte
 * aligned codes); elements 32 b .. 32 b + 31 of a row share scale c = scales[t, b], X = c - 127 the
 * smallest X >= -127 with max|x| <= 448 2^X (an all-zero block takes X = -127), and
 * codes = E4M3-RNE(x / 2^X): nothing saturates. A NaN or infinite element takes the NaN code and
 * leaves its block's other elements alone.
 *
 * D % 32 == 0, 32 <= D <= 2^24, 0 <= T < 2^31 (T = 0: nothing is done). `type` is the element type of x, y, dy, dx;
 * their rows are 16-byte aligned at pitches ld (elements, >= D).
 */
enum { ELMO_ACT_NONE = 0, ELMO_ACT_RELU = 1, ELMO_ACT_SILU = 2, ELMO_ACT_GELU = 3 };
/* Saves x [T, D]; with act != NONE also y = act(x) of the unrounded x, in the same pass (y nullable
 * only with NONE, where it must be NULL). relu(x) = max(x, 0); silu(x) = x / (1 + e^-x); gelu(x) =
 * x Phi(x), Phi the normal distribution function (no tanh approximation; results under 1e-37 may be 0, and so
 * may slopes below). y must not overlap x. */
int elmo_ckpt8_save(const void* x, int type, int64_t T, int D, int64_t ldx, int act, uint8_t* codes,
                    uint8_t* scales, void* y, int64_t ldy, void* stream);
/* The saved activations, x' [T, D]: exact in FP32 and BF16 (as far as the type's range goes), rounded in FP16. */
int elmo_ckpt8_load(const uint8_t* codes, const uint8_t* scales, int64_t T, int D, void* x, int type, int64_t ldx,
                    void* stream);
/* dx = dy act'(x') with the saved x' (relu'(0) = 0), act != NONE; dx = dy with equal pitches is allowed. */
int elmo_ckpt8_act_grad(const void* dy, int type, int64_t T, int D, int64_t lddy, int act, const uint8_t* codes,
                        const uint8_t* scales, void* dx, int64_t lddx, void* stream);
/* The weight gradient of a linear layer Y = X W^T from its saved input: dW [O, D] FP32 (row-major, 16-byte
 * aligned) = dY^T x', plus dW's old values if `accumulate` is nonzero. dY [T, O] BF16, 16-byte aligned rows
 * (O % 8 == 0, ldy % 8 == 0, ldy <= 2^23). Products of exact operands, binary32 sums in an order fixed by the shape.
 * T = 0 gives 0 (or leaves dW). The workspace holds the partial sums of split tokens. */
size_t elmo_ckpt8_weight_grad_workspace_bytes(int64_t T, int O, int D);
int elmo_ckpt8_weight_grad(const void* dY, int64_t ldy, const uint8_t* codes, const uint8_t* scales, int64_t T, int O,
                           int D, float* dW, int accumulate, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Log probabilities of given labels straight from features X and head weights W, without the logits
 * Z = X W^T ever being kept: the softmax cross entropy of a linear head over a large vocabulary.
 *
 *   X        [N, D], W [V, D] of element type `type` (BF16 or FP16), rows of adjacent elements at pitches
 *            ldx, ldw (elements, >= D, below 2^22 - 63); 16-byte aligned rows.
 *   ids      [N, M] int32, 0 <= M <= ELMO_MAX_GIVEN (NULL if M = 0); negative: no label (log probability 0 in
 *            any row); an id >= V gives NaN.
 *   logp     [N, M] FP32: (z[id] - row_max) - log_sum.
 *   row_max, log_sum  [N] FP32: max_v z_v and log sum_v e^(z_v - row_max); their sum is the log partition.
 * Products of exact operands, binary32 sums; logits below 2^126 in magnitude. A row of nothing but -inf logits has row_max
 * -inf, log_sum 0 and its labels' log probabilities -inf; a NaN or +inf logit makes log_sum and logp of its
 * row NaN (row_max skips NaN). Results repeat bit for bit on one device.
 * D % 32 == 0, 32 <= D <= ELMO_MAX_LINEAR_D; 1 <= V < 2^31, 0 <= N < 2^31 (N = 0: nothing is done), fewer than 2^30 tiles of
 * 64 x 64 logits (ELMO_ESHAPE). The workspace
 * takes 8 bytes for 128 logits (for 32 where there are few).
 */
#define ELMO_MAX_LINEAR_D 65536
size_t elmo_linear_logprobs_workspace_bytes(int64_t N, int64_t V, int D, int M);
int elmo_linear_logprobs(const void* X, const void* W, int type, int64_t N, int64_t V, int D, int64_t ldx, int64_t ldw,
                         const int32_t* ids, int M, float* logp, float* row_max, float* log_sum, void* workspace,
                         size_t workspace_bytes, void* stream);
/*
 * The gradients of the above with respect to X and W, from the upstream gradients dlogp [N, M] (NULL if
 * M = 0) and dlse [N] (nullable: of row_max + log_sum):
 *   G[n, v] = p_v (dlse - sum_j dlogp_j) + sum_{j : ids_j = v} dlogp_j;  dX = G W;  dW = G^T X.
 * row_max and log_sum are elmo_linear_logprobs' outputs for the same X and W. The vocabulary goes in pieces
 * of `chunk` labels (rounded up to a multiple of 256; 0: the library's choice, about 2^27 numbers of G, or 2^28 for N <=
 * 128): a piece's logits are computed again and G held in the workspace, the one rounding below 32 bits, relative to each
 * element: in X's type for a result of 16 bits, as the sum of two such numbers for a result in FP32, and for N <= 128; sums
 * are binary32. A label given more than once receives the sum of its gradients, a negative
 * id none. A row of nothing but -inf logits has G = 0; an id >= V makes G NaN in the whole row.
 *   dX       [N, D] of type `dx_type` (any), dW [V, D] of type `dw_type`, 16-byte aligned rows at pitches lddx,
 *            lddw; either may be NULL. accumulate: dW is added to, in binary32, and rounded once.
 * Neither overlaps another argument (dW is written while W is read). In FP16 an element of G is also off by up to 2^-39
 * of the largest |dlse| + 2 sum |dlogp| of a row. Probabilities below 2^-126 count as 0.
 * N = 0 leaves dW zero (or as it is with accumulate). Results repeat bit for bit on one device.
 * The workspace's size: need_dx, need_dw are 0 for a result that is not needed, 2 + its element type, or 1: any type.
 */
size_t elmo_linear_logprobs_backward_workspace_bytes(int64_t N, int64_t V, int D, int M, int64_t chunk, int need_dx,
                                                     int need_dw);
int elmo_linear_logprobs_backward(const void* X, const void* W, int type, int64_t N, int64_t V, int D, int64_t ldx,
                                  int64_t ldw, const int32_t* ids, int M, const float* row_max, const float* log_sum,
                                  const float* dlogp, const float* dlse, void* dX, int dx_type, int64_t lddx, void* dW,
                                  int dw_type, int64_t lddw, int accumulate, int64_t chunk, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * Products of rows held in 8-bit integers, with a scale for each row of both operands (each token, each
 * output channel): Y[n, v] = x_scales[n] w_scales[v] sum_k X[n, k] W[v, k]. The sum is exact; it is rounded to
 * binary32, multiplied by x_scales[n], then by w_scales[v], and rounded to `ytype`.
 *   X [N, D], W [L, D] int8 (any of -128 .. 127), row-major without gaps, 16-byte aligned; D % 64 == 0,
 *   64 <= D <= ELMO_MAX_I8_D. x_scales [N], w_scales [L] FP32. Y [N, L] of element type `ytype`, row n at Y + n ldy,
 *   any pitch and element alignment. 1 <= L < 2^31, 0 <= N < 2^31 (N = 0: nothing is done), fewer than 2^30
 *   tiles of 64 x 64 results. A NaN scale stays
 *   in its row or column. The workspace holds the sums of runs of K where there are few results; its size is 0 where none is
 *   needed (it may be NULL then), and for unsupported shapes.
 * elmo_i8_quantize makes such rows from x [N, D] (element type `type`, 16-byte aligned rows at pitch ldx):
 *   scale = max_k |x[k]| / 127, code = 127 x / max|x| to the nearest whole number, halves to the even one, of the
 *   exact quotient. A zero row has scale 0 and codes 0; a row with a NaN or an infinity has scale NaN and
 *   codes 0.
 */
#define ELMO_MAX_I8_D 65536
int elmo_i8_quantize(const void* x, int type, int64_t N, int D, int64_t ldx, int8_t* codes, float* scales, void* stream);
size_t elmo_i8_matmul_workspace_bytes(int64_t N, int64_t L, int D);
int elmo_i8_matmul(const int8_t* X, const float* x_scales, const int8_t* W, const float* w_scales, int64_t N, int64_t L,
                   int D, void* Y, int ytype, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Dropout from the generator of the stochastic rounding, with a mask that is never stored:
 *   y[t, d] = residual[t, d] + (kept ? x[t, d] 65536 / (65536 - limit) : 0), limit = floor(65536 p + 1/2);
 * element i = first + t D + d is kept if its 16 random bits are >= limit: Philox4x32-10 with key = `seed` and
 * counter (i >> 3, step), half (i & 1) of output word (i >> 1) & 3, as the weights' update draws (a call with
 * elmo_xmc_step's own seed and step shares its draws). In binary32, rounded once; dropped elements are 0
 * whatever they hold. The gradient with respect to x is the same call on dy without a residual.
 *   x, y, residual (nullable)  T rows of D elements of `type`, any pitch and element alignment. y = x or
 *            y = residual with equal pitches is allowed.
 *   p        0 <= p <= 1 (1: everything is dropped).
 *   step_at  device address of a number added to `step` when the work runs (NULL: none; 8-byte aligned): a
 *            recorded graph that counts it up draws a new mask at each replay.
 *   first    the index of x[0, 0]: parts of a batch draw what the whole would. first + T D <= 2^64 - 8.
 * 0 <= T < 2^31 (0: nothing is done), 1 <= D < 2^31. No workspace.
 */
int elmo_dropout(const void* x, int type, int64_t T, int64_t D, int64_t ldx, const void* residual, int64_t ldr, double p,
                 uint64_t seed, uint64_t step, const uint64_t* step_at, uint64_t first, void* y, int64_t ldy, void* stream);

/*
 * Test hook: the device codec, stochastic rounding and RNG applied elementwise to n elements.
 *   op 0  BF16 RNE encode:      in0 float[n]            -> out uint16[n]
 *   op 1  E4M3 RNE-sat encode:  in0 float[n]            -> out uint8[n]
 *   op 2  E4M3 decode:          in0 uint8[n]            -> out float[n]
 *   op 3  SR to BF16:           in0 float[n], in1 uint32 r[n] -> out uint16[n]
 *   op 4  SR to E4M3:           in0 float[n], in1 uint32 r[n] -> out uint8[n]
 *   op 5  RNG 16-bit draws:     r16(seed, step, idx0 + i), idx0 = *(const uint64_t*)in0 (HOST) -> out uint32[n]
 *   op 6  gradient code:        in0 float z[n], in1 uint32 y[n] -> out uint16[n] (BF16(sigmoid(z) - y))
 *   op 7  E4M3 -> BF16, 4 codes per word as the backward kernel decodes its weight tiles:
 *                               in0 uint32[n] -> out uint32[2n] (BF16 pairs of bytes 0,1 and 2,3)
 *   op 8  gradient, the forward's small-argument form (meant for |z| <= 2), binary32 before rounding:
 *                               in0 float z[n], in1 uint32 y[n] -> out float[n]
 *   op 9  gradient, the forward's split-exponent form (meant for |z| <= 80), binary32 before rounding:
 *                               in0 float z[n], in1 uint32 y[n] -> out float[n]
 *   op 10 SR to E2M1 (v already divided by its block scale): in0 float[n], in1 uint32 r[n] -> out uint8[n]
 *   op 11 MX block quantisation: in0 float t[32 n], in1 uint32 r[32 n] -> out uint8[33 n] (per block the
 *                               32 E2M1 codes, then the E8M0 scale code; 255 for a block with a NaN)
 *   op 12 E2M1 -> BF16 as the backward decodes MXFP4 weight tiles: in0 uint32 w[n] (8 codes, low
 *                               nibble first), in1 uint32 E8M0 scale code[n] -> out uint32[4 n] (BF16 pairs)
 *   op 13 one scaled MFMA in the forward's MXFP4 operand layout (E4M3 A, E2M1 B, E8M0 scales per
 *                               32-element block): in0 uint8[3200] = A codes [32][64], B codes [32][32]
 *                               (two per byte), A scales [32][2], B scales [32][2]; out float[1024] = C
 *                               [32][32] row-major; n must be 1
 *   op 14 the device's scaled FP4 conversion with stochastic rounding (a test hook for its rounding
 *                               rule): in0 float[2n] pairs, in1 uint32[2n] (random operand, scale
 *                               bits) per pair -> out uint32[n] (the two codes in byte 0)
 */
int elmo_numerics_probe(int op, const void* in0, const void* in1, void* out, int64_t n,
                        uint64_t seed, uint64_t step, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* ELMO_XMC_H */
