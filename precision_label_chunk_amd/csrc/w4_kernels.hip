// Products of a few BF16 feature rows with 4-bit weights: Y [N][L] = X [N][D] W^T, N <= 32.
//
// The weights are read once and are nearly all the traffic, so the kernels are built around feeding
// the HBM stream: every lane loads 16 bytes (32 codes of one label row) at a time, a wave 16 rows
// of 64 adjacent bytes, and the matrix cores do the sums, which leaves the vector units half an
// operation per weight (the decode to BF16, two codes at a time). The order of the features inside
// a product is free as long as both operands agree, so the 32 codes a lane holds go into four
// consecutive v_mfma_f32_16x16x32_bf16 as they lie: lane l holds label l % 16, and the features
// 32 (l / 16) + 8 i .. + 8 of the wave's 128 go into product i.
//   A: lane l holds row m = l % 16, k = 8 (l / 16) + e;  B: column l % 16, the same k;
//   C: lane l, register i holds column l % 16, row 4 (l / 16) + i.
//
// MXFP4 rows: the block's power-of-two scale is applied by the decode (exact in BF16), so row m of
// A is feature row m and the sums run over all of D.
//
// Integer codes with a scale (and zero point) per group: w = (c - z) s, s any BF16 number, which no
// exact BF16 weight holds. The codes 0..15 themselves are exact; the scale is applied to the
// binary32 sum of each 32 features. One product covers four such blocks (one per 16 lanes), kept
// apart by using A's sixteen rows for 4 feature rows x 4 blocks: row 4 n + b holds feature row n in
// block b's features and zeros elsewhere, so lane l's four results are the four blocks' sums of
// label l % 16 and feature row l / 16. The zero points take the features' own block sums, the same
// product against ones. A code byte c in 0..15 read as E4M3 is c 2^-9 (subnormals and the first
// binade have the same spacing), so the FP8 -> BF16 conversion with scale 2^9 decodes it.
#include "elem_types.hpp"
#include "step_kernels.hpp"

namespace elmo {

typedef int i32x4_a8 __attribute__((ext_vector_type(4), aligned(8)));
typedef int i32x2_a8 __attribute__((ext_vector_type(2), aligned(8)));

__device__ __forceinline__ f32x4_t mfma16(i32x4_t a, i32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                  0, 0, 0);
}

struct W4Args {
  const uint8_t* W; int64_t L; int D;
  int group; const uint16_t* scales; const uint8_t* zeros;
  const uint16_t* X; int N; int64_t ldx;
  void* Y; int ytype; int64_t ldy;
  int64_t tiles;                      // ceil(L / 16)
};

__device__ __forceinline__ void store_result(const W4Args& a, int64_t at, float v) {
  if (a.ytype == T_F32_) ElemF32::store((float*)a.Y + at, v);
  else if (a.ytype == T_BF16_) ElemBF16::store((uint16_t*)a.Y + at, v);
  else ElemF16::store((uint16_t*)a.Y + at, v);
}

// Sums the KS waves that share a tile through LDS (in the order of the waves) and hands each sum
// to `out(value index, sum)` in one of them. part: [KS][V][64] floats of this tile's waves.
template <int KS, int V, typename F>
__device__ __forceinline__ void join_slices(const float (&v)[V], float* part, int ks, int lane, F&& out) {
  if constexpr (KS == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) out(i, v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) part[(ks * V + i) * 64 + lane] = v[i];
    __syncthreads();
    for (int i = ks; i < V; i += KS) {
      float s = part[i * 64 + lane];
#pragma unroll
      for (int w = 1; w < KS; ++w) s += part[(w * V + i) * 64 + lane];
      out(i, s);
    }
  }
}

// ---- MXFP4 ---------------------------------------------------------------------------------------
// Block of WAVES waves: WAVES / KS groups of LT tiles (16 labels each), the KS waves of a group
// taking every KS-th unit of 256 features. NT tiles of 16 feature rows.
template <int NT, int LT, int KS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_w4_mx(W4Args a) {
  constexpr int V = LT * NT * 4;
  __shared__ float part[KS > 1 ? WAVES * V * 64 : 1];
  const int wave = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  const int ks = wave % KS, grp = wave / KS;
  const int col = lane & 15, q = lane >> 4;
  const int64_t tile0 = ((int64_t)blockIdx.x * (WAVES / KS) + grp) * LT;
  const int64_t rowb = (int64_t)a.D / 2 + a.D / 32;
  const uint8_t* row[LT];
#pragma unroll
  for (int t = 0; t < LT; ++t) {
    int64_t label = (tile0 + t) * 16 + col;
    if (label >= a.L) label = a.L - 1;                     // (read again, not written)
    row[t] = a.W + label * rowb;
  }
  const uint16_t* x[NT];
  bool has[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    has[j] = 16 * j + col < a.N;
    x[j] = a.X + (has[j] ? 16 * j + col : 0) * a.ldx + 32 * q;
  }
  f32x4_t acc[LT][NT];
#pragma unroll
  for (int t = 0; t < LT; ++t)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[t][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  const int units = a.D / 256;
  i32x4_t w[LT][2], wn[LT][2];
  i32x2_t sc[LT], sn[LT];
  auto load = [&](int u, i32x4_t (&wd)[LT][2], i32x2_t (&sd)[LT]) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < LT; ++t) {
      const uint8_t* p = row[t] + u * 128 + 16 * q;
      wd[t][0] = __builtin_nontemporal_load((const i32x4_a8*)p);
      wd[t][1] = __builtin_nontemporal_load((const i32x4_a8*)(p + 64));
      sd[t] = *(const i32x2_a8*)(row[t] + a.D / 2 + u * 8);
    }
  };
  int u = ks;
  if (u < units) load(u, w, sc);
  for (; u < units; u += KS) {
    if (u + KS < units) load(u + KS, wn, sn);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float scale[LT];
#pragma unroll
      for (int t = 0; t < LT; ++t) scale[t] = e8m0_to_f32((uint32_t)sc[t][s] >> (8 * q));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        i32x4_t xf[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          xf[j] = i32x4_t{0, 0, 0, 0};
          if (has[j]) xf[j] = *(const i32x4_t*)(x[j] + u * 256 + s * 128 + 8 * i);
        }
#pragma unroll
        for (int t = 0; t < LT; ++t) {
          const uint32_t c = (uint32_t)w[t][s][i];
          const i32x4_t b = {(int)fp4x2_to_bf16x2<0>(c, scale[t]), (int)fp4x2_to_bf16x2<1>(c, scale[t]),
                             (int)fp4x2_to_bf16x2<2>(c, scale[t]), (int)fp4x2_to_bf16x2<3>(c, scale[t])};
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[t][j] = mfma16(xf[j], b, acc[t][j]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < LT; ++t) { w[t][0] = wn[t][0]; w[t][1] = wn[t][1]; sc[t] = sn[t]; }
  }
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = acc[i / (4 * NT)][i / 4 % NT][i % 4];
  join_slices<KS, V>(v, part + (KS > 1 ? grp * KS * V * 64 : 0), ks, lane, [&](int i, float s) {
    const int n = 16 * (i / 4 % NT) + 4 * q + i % 4;
    const int64_t label = (tile0 + i / (4 * NT)) * 16 + col;
    if (n < a.N && label < a.L) store_result(a, n * a.ldy + label, s);
  });
}

// ---- integer codes with group scales -----------------------------------------------------------
// four features' order inside a lane's 8 is that of the decode (even, then odd)
__device__ __forceinline__ i32x4_t even_odd(i32x4_t d) {
  return i32x4_t{(int)__builtin_amdgcn_perm((uint32_t)d[1], (uint32_t)d[0], 0x05040100u),
                 (int)__builtin_amdgcn_perm((uint32_t)d[3], (uint32_t)d[2], 0x05040100u),
                 (int)__builtin_amdgcn_perm((uint32_t)d[1], (uint32_t)d[0], 0x07060302u),
                 (int)__builtin_amdgcn_perm((uint32_t)d[3], (uint32_t)d[2], 0x07060302u)};
}
__device__ __forceinline__ uint32_t code2(uint32_t bytes, bool hi) {
  return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)bytes, 512.0f, true))
            : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)bytes, 512.0f, false));
}
__device__ __forceinline__ i32x4_t codes8(uint32_t w) {
  const uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
  return i32x4_t{(int)code2(lo, false), (int)code2(lo, true), (int)code2(hi, false), (int)code2(hi, true)};
}

// the scales and zero points of the four 32-feature blocks of unit u (128 features) of a label row
template <int G>
__device__ __forceinline__ void load_groups(const W4Args& a, int64_t label, int u, float (&s)[4], float (&z)[4]) {
  const int64_t base = label * (a.D / G);
  const int last = a.D / G - 1;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    int g = (4 * u + b) / (G / 32);
    if (g > last) g = last;                                // (features past D are zeros)
    s[b] = bf16_to_f32(a.scales[base + g]);
    z[b] = a.zeros ? (float)a.zeros[base + g] : 8.0f;
  }
}

// As above, over units of 128 features; NQ quads of feature rows.
template <int G, int NQ, int LT, int KS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_w4_int(W4Args a) {
  constexpr int V = LT * NQ;
  __shared__ float part[KS > 1 ? WAVES * V * 64 : 1];
  const int wave = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  const int ks = wave % KS, grp = wave / KS;
  const int col = lane & 15, q = lane >> 4;
  const int64_t tile0 = ((int64_t)blockIdx.x * (WAVES / KS) + grp) * LT;
  int64_t label[LT];
#pragma unroll
  for (int t = 0; t < LT; ++t) {
    label[t] = (tile0 + t) * 16 + col;
    if (label[t] >= a.L) label[t] = a.L - 1;
  }
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  const int units = (a.D + 127) / 128;
  const i32x4_t ones = {0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80};
  for (int u = ks; u < units; u += KS) {
    const bool in = u * 128 + 32 * q < a.D;                // D is a multiple of 32: whole blocks
    i32x4_t w[LT];
    float s[LT][4], z[LT][4];
#pragma unroll
    for (int t = 0; t < LT; ++t) {
      w[t] = i32x4_t{0, 0, 0, 0};
      if (in) w[t] = __builtin_nontemporal_load((const i32x4_t*)(a.W + label[t] * (a.D / 2) + u * 64 + 16 * q));
      load_groups<G>(a, label[t], u, s[t], z[t]);
    }
    i32x4_t wb[LT][4];
#pragma unroll
    for (int t = 0; t < LT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) wb[t][i] = codes8((uint32_t)w[t][i]);
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      const int n = 4 * j + (col >> 2);
      const bool mine = in && (col & 3) == q && n < a.N;
      i32x4_t xf[4];
      f32x4_t xs = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xf[i] = i32x4_t{0, 0, 0, 0};
        if (mine) xf[i] = even_odd(*(const i32x4_t*)(a.X + n * a.ldx + u * 128 + 32 * q + 8 * i));
        xs = mfma16(xf[i], ones, xs);
      }
#pragma unroll
      for (int t = 0; t < LT; ++t) {
        f32x4_t c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) c = mfma16(xf[i], wb[t][i], c);
#pragma unroll
        for (int b = 0; b < 4; ++b)
          acc[t * NQ + j] = __builtin_fmaf(s[t][b], __builtin_fmaf(-z[t][b], xs[b], c[b]), acc[t * NQ + j]);
      }
    }
  }
  join_slices<KS, V>(acc, part + (KS > 1 ? grp * KS * V * 64 : 0), ks, lane, [&](int i, float s) {
    const int n = 4 * (i % NQ) + q;
    const int64_t lab = (tile0 + i / NQ) * 16 + col;
    if (n < a.N && lab < a.L) store_result(a, n * a.ldy + lab, s);
  });
}

// ---- launchers -------------------------------------------------------------------------------------
template <int NT, int LT, int KS, int WAVES>
static int go_mx(const W4Args& a, hipStream_t st) {
  const int64_t per = (int64_t)(WAVES / KS) * LT, blocks = (a.tiles + per - 1) / per;
  hipLaunchKernelGGL((k_w4_mx<NT, LT, KS, WAVES>), dim3((unsigned)blocks), dim3(64 * WAVES), 0, st, a);
  return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
}
template <int NT>
static int pick_mx(const W4Args& a, hipStream_t st) {
  const int units = a.D / 256;
  if (a.tiles >= 16 * device_cus() || units == 1) return go_mx<NT, 2, 1, 4>(a, st);
  if (a.tiles >= 4 * device_cus() || units < 8) return go_mx<NT, 1, 2, 4>(a, st);
  return go_mx<NT, 1, 8, 8>(a, st);
}

template <int G, int NQ, int LT, int KS, int WAVES>
static int go_int(const W4Args& a, hipStream_t st) {
  const int64_t per = (int64_t)(WAVES / KS) * LT, blocks = (a.tiles + per - 1) / per;
  hipLaunchKernelGGL((k_w4_int<G, NQ, LT, KS, WAVES>), dim3((unsigned)blocks), dim3(64 * WAVES), 0, st, a);
  return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
}
template <int G, int NQ>
static int pick_int(const W4Args& a, hipStream_t st) {
  const int units = (a.D + 127) / 128;
  if (a.tiles >= 16 * device_cus() || units < 4) return go_int<G, NQ, 1, 1, 4>(a, st);
  return go_int<G, NQ, 1, 8, 8>(a, st);
}
template <int G>
static int pick_rows(const W4Args& a, hipStream_t st) {
  if (a.N <= 4) return pick_int<G, 1>(a, st);
  if (a.N <= 16) return pick_int<G, 4>(a, st);
  return pick_int<G, 8>(a, st);
}

static int pick_format(const W4Args& a, int wdtype, hipStream_t st) {
  if (wdtype == W_MXFP4_) return a.N <= 16 ? pick_mx<1>(a, st) : pick_mx<2>(a, st);
  if (a.group == 32) return pick_rows<32>(a, st);
  if (a.group == 64) return pick_rows<64>(a, st);
  return pick_rows<128>(a, st);
}

int run_w4_matvec(const void* W, int wdtype, int64_t L, int D, int group, const uint16_t* scales, const uint8_t* zeros,
                  const void* X, int N, int64_t ldx, void* Y, int ytype, int64_t ldy, hipStream_t st) {
  W4Args a{};
  a.W = (const uint8_t*)W; a.L = L; a.D = D; a.group = group; a.scales = scales; a.zeros = zeros;
  a.X = (const uint16_t*)X; a.N = N; a.ldx = ldx; a.Y = Y; a.ldy = ldy;
  a.tiles = (L + 15) / 16;
  a.ytype = ytype;
  return pick_format(a, wdtype, st);
}

}  // namespace elmo
