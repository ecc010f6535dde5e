// Activations kept in 8 bits between the forward and the backward pass, and the two places where the
// backward uses them: the derivative of an elementwise activation, and the weight gradient of the
// linear layer behind it.
//
// Format (the layout of the MX weight formats, with 8-bit elements): 32 consecutive features of a
// token share one E8M0 scale 2^X, the smallest power of two with max |x| <= 448 2^X, and are stored
// as E4M3 to nearest even. The scale is taken from the elements themselves rather than rounded down
// as floor(log2 max |x|) - 8 would: that saturates blocks whose largest element is over 1.75 times
// its power of two, an error of up to 12.5% in the block's largest value; this costs the smallest
// elements of such a block one bit instead. Decoding is exact in BF16 (4 significant bits times a
// power of two), so that the matrix products read exact operands.
#include "elem_types.hpp"
#include "lm_kernels.hpp"

namespace elmo {

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3 };

// Phi(x) and e^(-x^2/2), the normal distribution and its unscaled density. With z = |x| / sqrt 2 and
// t = 1 / (1 + c z), erfc(z) / 2 = e^(-z^2) t P(t), P fitted to erfcx(z) / (2 t) over z <= 11 for the
// smallest relative error; the tail keeps its relative accuracy because nothing is subtracted from 1
// there. For FP32 outputs c = 0.3 and degree 8 (2.0e-8; in binary32 x Phi(x) is within 6e-7 relative down
// to x = -13), for 16-bit ones c = 0.5, degree 6 (1.7e-6, a two-hundredth of FP16's rounding) and a plain
// exponent (1.3e-5 at x = -13): the activation is as long as the memory traffic that hides it, and eight
// operations less.
template <bool FINE>
__device__ __forceinline__ void normal_parts(float x, float& cdf, float& dens) {
  float t, p;
  if constexpr (FINE) {
    t = __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fabsf(x), 0.2121320366859436f, 1.0f));
    p = -0.06477801501750946f;
    p = __builtin_fmaf(p, t, 0.2428685873746872f);
    p = __builtin_fmaf(p, t, -0.2563348710536957f);
    p = __builtin_fmaf(p, t, 0.274106502532959f);
    p = __builtin_fmaf(p, t, -0.047514792531728745f);
    p = __builtin_fmaf(p, t, 0.1075538918375969f);
    p = __builtin_fmaf(p, t, 0.07414305955171585f);
    p = __builtin_fmaf(p, t, 0.08536191284656525f);
    p = __builtin_fmaf(p, t, 0.08459370583295822f);
  } else {
    t = __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fabsf(x), 0.3535533845424652f, 1.0f));
    p = 0.04323947802186012f;
    p = __builtin_fmaf(p, t, -0.17534863948822021f);
    p = __builtin_fmaf(p, t, 0.19041365385055542f);
    p = __builtin_fmaf(p, t, 0.021891044452786446f);
    p = __builtin_fmaf(p, t, 0.13965976238250732f);
    p = __builtin_fmaf(p, t, 0.13899248838424683f);
    p = __builtin_fmaf(p, t, 0.14115135371685028f);
  }
  if constexpr (FINE) {
    // y = -x^2 log2(e) / 2 is rounded three times (the square, the constant, their product), which alone
    // is x^2 / 2 times as large in the result: what they left out, dy, is put back as 1 + dy ln 2
    const float c = __builtin_fminf(__builtin_fabsf(x), 16.0f), s = c * c, y = s * -0.72134751081466675f;
    float dy = __builtin_fmaf(s, -0.72134751081466675f, -y);
    dy = __builtin_fmaf(__builtin_fmaf(c, c, -s), -0.72134751081466675f, dy);
    dy = __builtin_fmaf(s, -9.62981517e-09f, dy);
    dens = __builtin_amdgcn_exp2f(y);
    dens = __builtin_fmaf(dens, dy * 0.69314718f, dens);
  } else {
    const float u = x * 0.84932180028801904f;              // sqrt(log2(e) / 2)
    dens = __builtin_amdgcn_exp2f(-(u * u));
  }
  const float half = t * p * dens;
  cdf = x < 0.0f ? half : 1.0f - half;
}
// sigma(x) = a (a r) and 1 - sigma(x) = q, without cancellation: with e = e^(-|x|) and r = 1 / (1 + e),
// sigma is r or e r and its complement the other. Below 0, e is split into two factors a = e^(-|x|/2),
// so that x sigma(x) keeps its value down to the smallest results (x = -100) where e leaves the
// normal range.
struct Sigmoid { float a, ar, q; };
__device__ __forceinline__ Sigmoid sigmoid_parts(float x) {
  const float h = __builtin_amdgcn_exp2f(__builtin_fabsf(x) * -0.72134752044448170f);
  const float e = h * h, r = __builtin_amdgcn_rcpf(1.0f + e);
  const bool neg = x < 0.0f;
  const float a = neg ? h : 1.0f;
  return Sigmoid{a, a * r, neg ? r : e * r};
}

template <int ACT, bool FINE>
__device__ __forceinline__ float act_value(float x) {
  if constexpr (ACT == ACT_RELU) return x < 0.0f ? 0.0f : x;           // (NaN stays)
  if constexpr (ACT == ACT_SILU) {
    const Sigmoid s = sigmoid_parts(x);
    return (x * s.a) * s.ar;
  }
  if constexpr (ACT == ACT_GELU) {
    float cdf, dens;
    normal_parts<FINE>(x, cdf, dens);
    return x * cdf;
  }
  return x;
}
template <int ACT, bool FINE>
__device__ __forceinline__ float act_slope(float x) {
  if constexpr (ACT == ACT_RELU) return x > 0.0f ? 1.0f : x <= 0.0f ? 0.0f : x;
  if constexpr (ACT == ACT_SILU) {
    const Sigmoid s = sigmoid_parts(x);
    return s.a * (s.ar * __builtin_fmaf(x, s.q, 1.0f));
  }
  if constexpr (ACT == ACT_GELU) {
    float cdf, dens;
    normal_parts<FINE>(x, cdf, dens);
    return __builtin_fmaf(x * 0.39894228040143268f, dens, cdf);        // 1 / sqrt(2 pi)
  }
  return 1.0f;
}

typedef __attribute__((ext_vector_type(2))) short s16x2_t;

// 8 consecutive elements at p, 16-byte aligned
template <typename E>
__device__ __forceinline__ void load8(const typename E::raw* p, float (&f)[8]) {
  E::widen(__builtin_nontemporal_load((const i32x4_t*)p), f);
  if constexpr (E::VEC == 4) E::widen(__builtin_nontemporal_load((const i32x4_t*)p + 1), f + 4);
}
// Non-temporal stores only where each covers whole lines: FP32 rows take two stores per thread, 32 bytes
// apart (16384 x 4096 restored in 56 us with plain stores, 97 with non-temporal ones)
template <typename E>
__device__ __forceinline__ void store8(typename E::raw* p, const float (&f)[8]) {
  if constexpr (E::VEC == 4) {
    *(i32x4_t*)p = E::narrow(f);
    *((i32x4_t*)p + 1) = E::narrow(f + 4);
  } else {
    __builtin_nontemporal_store(E::narrow(f), (i32x4_t*)p);
  }
}
// the 8 elements that 8 codes stand for; the conversion takes a scale's exponent field alone, which
// means in E8M0 what it means there (0: 2^-127, 255: NaN)
__device__ __forceinline__ void decode8(i32x2_t c, uint32_t scale_code, float (&f)[8]) {
  const float scale = u2f(scale_code << 23);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = c[h];
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, false);
    const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, true);
    f[4 * h] = a[0]; f[4 * h + 1] = a[1];
    f[4 * h + 2] = b[0]; f[4 * h + 3] = b[1];
  }
}

// the largest magnitude of a block's bits to its scale code X + 127: floor(log2 a) - 8 + 127, one
// more where the fraction is over 1.75; at least 0 (2^-127, also for a block of zeros)
__device__ __forceinline__ uint32_t block_scale_code(uint32_t a) {
  const int c = (int)(a >> 23) - 8 + ((a & 0x7fffffu) > 0x600000u ? 1 : 0);
  return c < 0 ? 0u : (uint32_t)c;
}

struct Ckpt8Args {
  const void* in; int64_t ldin;                 // x, or dy
  void* out; int64_t ldout;                     // y, dx or the restored activations (nullable in save)
  uint8_t* codes; uint8_t* scales;
  int64_t n8; int D;                            // vectors of 8 features
};

// start of vector i in a matrix of row pitch ld
__device__ __forceinline__ int64_t vec_at(int64_t i, int D, int64_t ld) {
  if (ld == D) return 8 * i;
  const int64_t row = i / (D / 8);
  return row * ld + 8 * (i - row * (D / 8));
}

// Elementwise, bound by HBM: each thread takes 8 features (one 16-byte load of a 16-bit type), the
// four threads of a block of 32 share their largest magnitude. 16384 x 4096 BF16 with gelu in 53 us
// (6.4 TB/s), relu 52, kept alone 37 (5.5 TB/s).
template <typename E, int ACT, bool OUT>
__global__ __launch_bounds__(256) void k_ckpt8_save(Ckpt8Args a) {
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < a.n8; i += (int64_t)gridDim.x * 256) {
    float f[8];
    load8<E>((const typename E::raw*)a.in + vec_at(i, a.D, a.ldin), f);
    uint32_t top = 0;                                       // as whole numbers: signalling NaNs upset v_max_f32
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t m = f2u(f[e]) & 0x7fffffffu;
      top = m > top ? m : top;
    }
    if (__builtin_expect(top >= 0x7f800000u, 0)) {          // infinity and NaN set no scale
      top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t m = f2u(f[e]) & 0x7fffffffu;
        top = m > top && m < 0x7f800000u ? m : top;
      }
    }
    const uint32_t t1 = (uint32_t)__shfl_xor((int)top, 1);
    top = t1 > top ? t1 : top;
    const uint32_t t2 = (uint32_t)__shfl_xor((int)top, 2);
    top = t2 > top ? t2 : top;
    const uint32_t code = block_scale_code(top);
    // the conversion divides by the scale (its exponent field: 0 for 2^-127), exactly, and rounds to nearest
    // even; no finite element is over 448, and infinity and NaN both give the NaN code
    const float scale = u2f(code << 23);
    i32x2_t c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s16x2_t w = {0, 0};
      w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, f[4 * h], f[4 * h + 1], scale, false);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, f[4 * h + 2], f[4 * h + 3], scale, true);
      c[h] = __builtin_bit_cast(int, w);
    }
    ((i32x2_t*)a.codes)[i] = c;
    if ((i & 3) == 0) a.scales[i >> 2] = (uint8_t)code;
    if constexpr (OUT) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = act_value<ACT, E::VEC == 4>(f[e]);
      store8<E>((typename E::raw*)a.out + vec_at(i, a.D, a.ldout), f);
    }
  }
}

template <typename E>
__global__ __launch_bounds__(256) void k_ckpt8_load(Ckpt8Args a) {
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < a.n8; i += (int64_t)gridDim.x * 256) {
    float f[8];
    decode8(__builtin_nontemporal_load((const i32x2_t*)a.codes + i), a.scales[i >> 2], f);
    store8<E>((typename E::raw*)a.out + vec_at(i, a.D, a.ldout), f);
  }
}

// dx = dy act'(x) with x from its 8 bits; dx may be dy's own memory. Bound by HBM: 16384 x 4096 BF16 in
// 55 us with relu (6.2 TB/s), 57 with silu and 59 with gelu (5.7), whose arithmetic is not all hidden.
template <typename E, int ACT>
__global__ __launch_bounds__(256) void k_ckpt8_act_grad(Ckpt8Args a) {
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < a.n8; i += (int64_t)gridDim.x * 256) {
    float f[8], d[8];
    load8<E>((const typename E::raw*)a.in + vec_at(i, a.D, a.ldin), d);
    decode8(__builtin_nontemporal_load((const i32x2_t*)a.codes + i), a.scales[i >> 2], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] *= act_slope<ACT, E::VEC == 4>(f[e]);
    store8<E>((typename E::raw*)a.out + vec_at(i, a.D, a.ldout), d);
  }
}

// ---- weight gradient -------------------------------------------------------------------------------
// dW [O][D] = dY^T X over T tokens, dY BF16 [T][O], X the 8-bit form [T][D]; FP32 sums.
//
// Both operands have the contraction (tokens) as their rows, so both come out of LDS through the
// transposing reads (ds_read_b64_tr_b16). A block of 4 waves (2 x 2) owns a tile of 64 MF x 64 NF
// of dW, each wave MF x NF products of 32 x 32; a stage holds BK tokens of both operands as BF16,
// the codes decoded on their way into LDS (half an operation per code, shared by the whole tile).
// Two LDS buffers and the next one or two stages' loads in registers: one barrier per stage. Rows are
// padded by 64 bytes, so that the four token rows of a transposing read cover all 64 banks (no
// conflicts counted). Bound by latency: one wave per SIMD has nothing to run while it waits. 16384
// tokens, 2048 x 4096, the join included: 269 us on inputs used again and 294 (936 TFLOP/s) on inputs
// that change from call to call, where the library's BF16 product of the decoded operands, timed in
// turn with it, takes 245 and 255. (The product alone 271, the join 18; the first dozen launches after an
// idle time take 300 to 345.) On changing inputs the matrix cores are busy 41% of the cycles, LDS
// 21%, and the waves spend 39% of theirs waiting for data or at the barrier.
// Few tiles split the tokens over `segs` blocks, whose partial tiles k_wgrad_join adds in order.
constexpr int WG_BK = 32;
struct WgradArgs {
  const uint16_t* dY; int64_t ldy;
  const uint8_t *codes, *scales;
  int64_t T; int O, D;
  float* dW; int accumulate;
  int segs; int64_t per;                        // tokens per segment, a multiple of WG_BK
  float* part;                                  // [segs][O][D]
  int tiles, tiles_d;
};

template <int MF, int NF, int AHEAD>
__global__ __launch_bounds__(256) void k_ckpt8_wgrad(WgradArgs a) {
  constexpr int BM = 64 * MF, BN = 64 * NF;
  constexpr int PA = BM + 32, PB = BN + 32;               // LDS row pitch (elements)
  constexpr int NA = WG_BK * BM / 8 / 256;                // 16-byte vectors of dY per thread and stage
  constexpr int NB = WG_BK * BN / 8 / 256;                // 8-code vectors per thread and stage
  __shared__ __attribute__((aligned(16))) uint16_t la[2][WG_BK * PA];
  __shared__ __attribute__((aligned(16))) uint16_t lb[2][WG_BK * PB];
  const int tid = (int)threadIdx.x, wave = tid >> 6, lane = tid & 63;
  // Blocks go to the 8 XCDs in turn; each XCD gets a run of (segment, tile) in that order, so that the
  // tiles that read a segment's tokens share an L2 (16384 tokens, 768 x 768 with the large tile: 73 -> 48 us)
  const int n = (int)gridDim.x, xcd = (int)blockIdx.x & 7, run = n / 8, more = n % 8;
  const int id = xcd * run + (xcd < more ? xcd : more) + (int)(blockIdx.x >> 3);
  const int seg = id / a.tiles, tile = id % a.tiles;
  const int o0 = tile / a.tiles_d * BM, d0 = tile % a.tiles_d * BN;
  const int64_t t0 = seg * a.per;
  const int64_t t1 = t0 + a.per < a.T ? t0 + a.per : a.T;

  // A thread's vectors of a stage lie a fixed number of token rows apart: one offset per operand is
  // held, the others are formed at each fetch. The buffers end with the segment's last token, so that rows past it read zeros;
  // columns past O or D read other elements of the matrix and reach only results that are not stored.
  constexpr int KA = 256 / (BM / 8), KB = 256 / (BN / 8);  // token rows between a thread's vectors
  const int ka = tid / (BM / 8), ca = tid % (BM / 8) * 8, kb = tid / (BN / 8), cb = tid % (BN / 8) * 8;
  const int sd = a.D / 32, lda = (int)a.ldy * 2;
  const int offa = ka * lda + 2 * ca, offb = kb * a.D + cb, offs = kb * sd + cb / 32;
  i32x4_t ra[AHEAD][NA];
  i32x2_t rb[AHEAD][NB];
  uint32_t rs[AHEAD][NB];
  auto fetch = [&](int64_t t, int r) __attribute__((always_inline)) {
    const int rows = t1 - t > 0 ? (int)(t1 - t < 2 * WG_BK ? t1 - t : 2 * WG_BK) : 0;   // (a stage reads WG_BK)
    const auto bufa = buffer_rsrc(a.dY + t * a.ldy + o0, rows ? (rows - 1) * lda + 2 * (a.O - o0) : 0);
    const auto bufb = buffer_rsrc(a.codes + t * a.D + d0, rows ? rows * a.D - d0 : 0);
    const auto bufs = buffer_rsrc(a.scales + t * sd + d0 / 32, rows ? rows * sd - d0 / 32 : 0);
    int oa = offa, ob = offb, os = offs;
    asm volatile("" : "+v"(oa), "+v"(ob), "+v"(os));        // (not hoisted: a register each across the loop)
#pragma unroll
    for (int v = 0; v < NA; ++v) ra[r][v] = buffer_load16(bufa, oa + v * KA * lda);
#pragma unroll
    for (int v = 0; v < NB; ++v) {
      rb[r][v] = __builtin_amdgcn_raw_buffer_load_b64(bufb, ob + v * KB * a.D, 0, 0);
      rs[r][v] = __builtin_amdgcn_raw_buffer_load_b8(bufs, os + v * KB * sd, 0, 0);
    }
  };
  auto put = [&](int b, int r) __attribute__((always_inline)) {
#pragma unroll
    for (int v = 0; v < NA; ++v) *(i32x4_t*)&la[b][(ka + v * KA) * PA + ca] = ra[r][v];
#pragma unroll
    for (int v = 0; v < NB; ++v) {
      const float s = u2f(rs[r][v] << 23);                  // (the conversion takes the exponent field alone)
      i32x4_t w;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int q = rb[r][v][h];
        w[2 * h] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, s, false));
        w[2 * h + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, s, true));
      }
      *(i32x4_t*)&lb[b][(kb + v * KB) * PB + cb] = w;
    }
  };

  f32x16_t acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  // lane's place in a transposing read: group g of 16 lanes takes columns 16 (g & 1) .. + 16 and rows
  // 8 (g >> 1) .. + 4 (then + 4 .. + 8); lane j of it supplies row j / 4, columns 4 (j % 4) .. + 4
  const int g = lane >> 4, j16 = lane & 15;
  const int mo = (wave >> 1) * 32 * MF + 16 * (g & 1) + 4 * (j16 & 3);
  const int no = (wave & 1) * 32 * NF + 16 * (g & 1) + 4 * (j16 & 3);
  const int ko = 8 * (g >> 1) + (j16 >> 2);

  s16x8_t fa[2][MF], fb[2][NF];
  auto frags = [&](int b, int kk, int f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const uint16_t* p = &la[b][(kk + ko) * PA + mo + 32 * i];
      fa[f][i] = join(lds_read_tr16(p), lds_read_tr16(p + 4 * PA));
    }
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const uint16_t* p = &lb[b][(kk + ko) * PB + no + 32 * j];
      fb[f][j] = join(lds_read_tr16(p), lds_read_tr16(p + 4 * PB));
    }
  };
  auto products = [&](int f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = mfma_bf16(fa[f][i], fb[f][j], acc[i][j]);
  };

  // Stage s: the second half's fragments are read under the first half's products, the next stage goes
  // to LDS and the one AHEAD stages later is fetched into its registers; behind the barrier the next
  // stage's first fragments are read under the second half's products. (fetch and put past the last
  // stage move zeros.)
  auto stage = [&](int64_t t, auto b) __attribute__((always_inline)) {
    const int B = b, RS = AHEAD == 2 ? B ^ 1 : 0;
    frags(B, 16, 1);
    products(0);
    put(B ^ 1, RS);
    fetch(t + (AHEAD + 1) * WG_BK, RS);
    // one product, then a share of the rest: an LDS read, conversions, an LDS write, a load
#pragma unroll
    for (int i = 0; i < MF * NF; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2 * (MF + NF) / (MF * NF) > 0 ? 2 * (MF + NF) / (MF * NF) : 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
      __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
    __syncthreads();
    frags(B ^ 1, 0, 0);
    products(1);
#pragma unroll
    for (int i = 0; i < MF * NF; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
  };
  fetch(t0, 0);
  put(0, 0);
  fetch(t0 + WG_BK, AHEAD - 1);                             // (AHEAD = 2: stage s in registers s & 1)
  if constexpr (AHEAD == 2) fetch(t0 + 2 * WG_BK, 0);
  __syncthreads();
  frags(0, 0, 0);
  if constexpr (AHEAD == 2) {                               // (the register sets named at compile time)
    for (int64_t t = t0; t < t1; t += 2 * WG_BK) {
      stage(t, std::integral_constant<int, 0>{});
      if (t + WG_BK < t1) stage(t + WG_BK, std::integral_constant<int, 1>{});
    }
  } else {
    int b = 0;
    for (int64_t t = t0; t < t1; t += WG_BK, b ^= 1) stage(t, b);
  }

  float* out = a.segs > 1 ? a.part + (int64_t)seg * a.O * a.D : a.dW;
  const bool add = a.segs == 1 && a.accumulate;
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int o = o0 + ((wave >> 1) * MF + i) * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
        const int d = d0 + ((wave & 1) * NF + j) * 32 + (lane & 31);
        if (o < a.O && d < a.D) {
          float* q = out + (int64_t)o * a.D + d;
          *q = add ? *q + acc[i][j][r] : acc[i][j][r];
        }
      }
}

// dW = (accumulate ? dW : 0) + the segments' partials. Thread (x, y) of a block of 64 x 4 sums the
// partials y, y + 4, .. of vector x; the four sums are added in the order of y.
__global__ __launch_bounds__(256) void k_wgrad_join(const float* part, float* dW, int64_t n4, int segs, int accumulate) {
  __shared__ f32x4_t sums[4][64];
  const int x = (int)threadIdx.x & 63, y = (int)threadIdx.x >> 6;
  for (int64_t i0 = blockIdx.x * (int64_t)64; i0 < n4; i0 += (int64_t)gridDim.x * 64) {
    const int64_t i = i0 + x;
    f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (i < n4) {
#pragma unroll 4
      for (int g = y; g < segs; g += 4) s += ((const f32x4_t*)part)[g * n4 + i];
    }
    sums[y][x] = s;
    __syncthreads();
    if (y == 0 && i < n4) {
      s += sums[1][x];
      s += sums[2][x];
      s += sums[3][x];
      if (accumulate) s += ((const f32x4_t*)dW)[i];
      ((f32x4_t*)dW)[i] = s;
    }
    __syncthreads();
  }
}

// ---- launchers -------------------------------------------------------------------------------------
static unsigned grid_of(int64_t n) {
  const int64_t want = (n + 255) / 256, cap = 256 * (int64_t)device_cus();
  return (unsigned)(want < cap ? want : cap);
}
#define ELMO_LAUNCH(kernel, n, st, ...)                                        \
  hipLaunchKernelGGL((kernel), dim3(grid_of(n)), dim3(256), 0, st, __VA_ARGS__)

template <typename E>
static void save_as(const Ckpt8Args& a, int act, hipStream_t st) {
  if (!a.out) ELMO_LAUNCH((k_ckpt8_save<E, ACT_NONE, false>), a.n8, st, a);
  else if (act == ACT_RELU) ELMO_LAUNCH((k_ckpt8_save<E, ACT_RELU, true>), a.n8, st, a);
  else if (act == ACT_SILU) ELMO_LAUNCH((k_ckpt8_save<E, ACT_SILU, true>), a.n8, st, a);
  else ELMO_LAUNCH((k_ckpt8_save<E, ACT_GELU, true>), a.n8, st, a);
}
template <typename E>
static void grad_as(const Ckpt8Args& a, int act, hipStream_t st) {
  if (act == ACT_RELU) ELMO_LAUNCH((k_ckpt8_act_grad<E, ACT_RELU>), a.n8, st, a);
  else if (act == ACT_SILU) ELMO_LAUNCH((k_ckpt8_act_grad<E, ACT_SILU>), a.n8, st, a);
  else ELMO_LAUNCH((k_ckpt8_act_grad<E, ACT_GELU>), a.n8, st, a);
}

int run_ckpt8_save(const void* x, int type, int64_t T, int D, int64_t ldx, int act, uint8_t* codes, uint8_t* scales,
                   void* y, int64_t ldy, hipStream_t st) {
  Ckpt8Args a{};
  a.in = x; a.ldin = ldx; a.out = y; a.ldout = ldy; a.codes = codes; a.scales = scales; a.n8 = T * (D / 8); a.D = D;
  if (type == T_F32_) save_as<ElemF32>(a, act, st);
  else if (type == T_BF16_) save_as<ElemBF16>(a, act, st);
  else save_as<ElemF16>(a, act, st);
  return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
}

int run_ckpt8_load(const uint8_t* codes, const uint8_t* scales, int64_t T, int D, void* x, int type, int64_t ldx,
                   hipStream_t st) {
  Ckpt8Args a{};
  a.out = x; a.ldout = ldx; a.codes = const_cast<uint8_t*>(codes); a.scales = const_cast<uint8_t*>(scales);
  a.n8 = T * (D / 8); a.D = D;
  if (type == T_F32_) ELMO_LAUNCH(k_ckpt8_load<ElemF32>, a.n8, st, a);
  else if (type == T_BF16_) ELMO_LAUNCH(k_ckpt8_load<ElemBF16>, a.n8, st, a);
  else ELMO_LAUNCH(k_ckpt8_load<ElemF16>, a.n8, st, a);
  return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
}

int run_ckpt8_act_grad(const void* dy, int type, int64_t T, int D, int64_t lddy, int act, const uint8_t* codes,
                       const uint8_t* scales, void* dx, int64_t lddx, hipStream_t st) {
  Ckpt8Args a{};
  a.in = dy; a.ldin = lddy; a.out = dx; a.ldout = lddx;
  a.codes = const_cast<uint8_t*>(codes); a.scales = const_cast<uint8_t*>(scales); a.n8 = T * (D / 8); a.D = D;
  if (type == T_F32_) grad_as<ElemF32>(a, act, st);
  else if (type == T_BF16_) grad_as<ElemBF16>(a, act, st);
  else grad_as<ElemF16>(a, act, st);
  return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
}

// Tile (128 x 128 or 256 x 256) and number of token segments by the time they are expected to take, in
// nanoseconds: a block's fixed part, its stages at the rate that one or several blocks per CU reach,
// and the join's launch and traffic (coefficients fitted to timings between 64 x 64 and 4096 x 4096).
// The large tile reads LDS half as often per product, the small one fills the device with less
// splitting: 16384 tokens (the same for every call) take 265 us with 256 x 256 and 324 with 128 x 128
// at 2048 x 4096, and 44 against 37 at 768 x 768.
WgradLayout wgrad_layout(int64_t T, int O, int D) {
  const int cus = device_cus();
  WgradLayout best{};
  double least = 0.0;
  for (int big = 0; big < 2; ++big) {
    const int tile = big ? 256 : 128;
    const int64_t to = (O + tile - 1) / tile, td = (D + tile - 1) / tile, tiles = to * td;
    const int64_t stages = (T + WG_BK - 1) / WG_BK;
    for (int64_t segs = 1; segs <= 256 && (segs == 1 || (segs <= stages && tiles * segs <= 4 * cus)); ++segs) {
      const int64_t per = (stages + segs - 1) / segs, used = per ? (stages + per - 1) / per : 1;
      if (used != segs && segs > 1) continue;
      const int64_t blocks = tiles * segs, most = (blocks + cus - 1) / cus;   // blocks on the fullest CU
      double ns;
      if (big) ns = 9000.0 + (double)most * per * 1000.0;
      else ns = 5000.0 + (double)(most / 2) * per * 640.0 + (double)(most % 2) * per * 530.0;
      if (segs > 1) ns += 3000.0 + (double)segs * O * D * (8.0 / 6000.0);
      if (least == 0.0 || ns < least) {
        least = ns;
        best.big = big; best.tiles_o = (int)to; best.tiles_d = (int)td; best.segs = (int)segs; best.per = per * WG_BK;
      }
    }
  }
  if (best.per < WG_BK) best.per = WG_BK;
  best.total = best.segs > 1 ? (size_t)best.segs * O * D * 4 : 256;
  return best;
}

int run_ckpt8_wgrad(const void* dY, int64_t ldy, const uint8_t* codes, const uint8_t* scales, int64_t T, int O, int D,
                    float* dW, int accumulate, const WgradLayout& s, void* workspace, hipStream_t st) {
  WgradArgs a{};
  a.dY = (const uint16_t*)dY; a.ldy = ldy; a.codes = codes; a.scales = scales; a.T = T; a.O = O; a.D = D;
  a.dW = dW; a.accumulate = accumulate; a.segs = s.segs; a.per = s.per; a.part = (float*)workspace; a.tiles_d = s.tiles_d;
  a.tiles = s.tiles_o * s.tiles_d;
  const dim3 grid((unsigned)((int64_t)s.tiles_o * s.tiles_d * s.segs));
  if (s.big)
    hipLaunchKernelGGL((k_ckpt8_wgrad<4, 4, 1>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_ckpt8_wgrad<2, 2, 2>), grid, dim3(256), 0, st, a);
  if (hipGetLastError() != hipSuccess) return ELMO_EHIP_;
  if (s.segs > 1) {
    const int64_t n4 = (int64_t)O * D / 4;
    ELMO_LAUNCH(k_wgrad_join, 4 * n4, st, (const float*)workspace, dW, n4, s.segs, accumulate);
    if (hipGetLastError() != hipSuccess) return ELMO_EHIP_;
  }
  return ELMO_OK_;
}

}  // namespace elmo
