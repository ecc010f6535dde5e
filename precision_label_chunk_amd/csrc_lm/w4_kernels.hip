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
// MXFP4 rows: the block's power-of-two scale is applied by the decode (exact in BF16 below 2^128, infinite
// from there), so row m of A is feature row m and the sums run over all of D.
//
// Integer codes with a scale (and zero point) per group: w = (c - z) s, s any BF16 number, which no
// exact BF16 weight holds. The codes 0..15 themselves are exact; the scale is applied to the
// binary32 sum of each group, the zero point to the features' own group sums (formed once per
// block). The 128 features of a wave's load are four blocks of 32, one per 16 lanes, and their sums
// have to stay apart down to the group size:
//   N <= 4: A's sixteen rows are 4 feature rows x 4 blocks, row 4 n + b holding feature row n in
//     block b's features and zeros elsewhere; the codes go into the products as they lie, and lane l
//     ends with the four block sums of label l % 16 and feature row l / 16.
//   N > 4: the codes are transposed between the four lanes of a label (two permlane32_swap, two
//     permlane16_swap per 32 codes), so that product b holds block b alone and A's rows are sixteen
//     feature rows: a quarter of the products and LDS reads of the first form at N = 16.
// A code byte c in 0..15 read as E4M3 is c 2^-9 (subnormals and the first binade have the same
// spacing), so the FP8 -> BF16 conversion with scale 2^9 decodes it.
#include "elem_types.hpp"
#include "lm_kernels.hpp"

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
  int64_t tile0;                      // the launch's first tile (k_w4_int_deep)
  // the panel of D that a launch takes, in the kernel's units of features: rows of larger products do
  // not fit LDS at once, and their FP32 results are summed panel by panel
  int unit0, units, add;
};

__device__ __forceinline__ void store_result(const W4Args& a, int64_t at, float v) {
  if (a.ytype == T_F32_) ElemF32::store((float*)a.Y + at, a.add ? ((const float*)a.Y)[at] + v : v);
  else if (a.ytype == T_BF16_) ElemBF16::store((uint16_t*)a.Y + at, v);
  else ElemF16::store((uint16_t*)a.Y + at, v);
}

__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0x0f70);                      // vmcnt(0), the other counters untouched
  __builtin_amdgcn_sched_barrier(0);
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
// Units of 256 features: 2 x 16 bytes of codes and 8 scale bytes per lane and tile of 16 labels.
struct MxUnit { i32x4_t w[2]; i32x2_t s; };

__device__ __forceinline__ const uint8_t* mx_row(const W4Args& a, int64_t tile, int col) {
  int64_t label = tile * 16 + col;
  if (label >= a.L) label = a.L - 1;                       // (read again, not written)
  return a.W + label * ((int64_t)a.D / 2 + a.D / 32);
}
__device__ __forceinline__ void load_unit(const W4Args& a, const uint8_t* row, int u, int q, MxUnit& m) {
  const uint8_t* p = row + u * 128 + 16 * q;
  m.w[0] = *(const i32x4_a8*)p;
  m.w[1] = *(const i32x4_a8*)(p + 64);
  m.s = *(const i32x2_a8*)(row + a.D / 2 + u * 8);
}
// byte q of a dword of E8M0 codes as the scale operand of the FP4 conversion, which takes a binary32
// number's exponent field alone: 0 stands for 2^-127 and 255 for NaN there, as in E8M0
__device__ __forceinline__ float mx_scale(int s, int q) { return u2f((((uint32_t)s >> (8 * q)) & 0xffu) << 23); }
__device__ __forceinline__ i32x4_t mx_decode8(uint32_t c, float scale) {
  return i32x4_t{(int)fp4x2_to_bf16x2<0>(c, scale), (int)fp4x2_to_bf16x2<1>(c, scale), (int)fp4x2_to_bf16x2<2>(c, scale),
                 (int)fp4x2_to_bf16x2<3>(c, scale)};
}
// the sums of C: registers i hold feature rows 4 q + i of label col
__device__ __forceinline__ void store_tile(const W4Args& a, int64_t tile, int n0, int col, int q, f32x4_t acc) {
  const int64_t label = tile * 16 + col;
  if (label >= a.L) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + 4 * q + i;
    if (n < a.N) store_result(a, n * a.ldy + label, acc[i]);
  }
}

// D <= 256 UNITS and N <= 16: the feature rows stay in registers, 32 per unit, for all the tiles a wave
// takes, and the loop reads nothing but weights, a whole tile (adjacent rows) at a time. The next
// tile's codes are loaded before the present one's products.
// Bound by HBM: 3M x 768 labels with one row in 222 us (5.6 TB/s), with 16 rows in 302 (4.7 TB/s: the
// results, 64 bytes to a row and tile, are written slower than weights are read); 131072 x 768 with
// one row in 13 us (4.1 TB/s; 11 where the 53 MB of weights are still in the last-level cache). Rows in LDS instead take 338 us against 304 at 3M x 768 with 16 rows,
// the simple form that reads them again for every tile 640; non-temporal loads of the weights 379 against
// 322 with plain ones (on an earlier form): adjacent rows share cache lines.
template <int UNITS>
__global__ __launch_bounds__(256) void k_w4_mx_regs(W4Args a) {
  const int lane = (int)threadIdx.x & 63, col = lane & 15, q = lane >> 4;
  const int64_t step = (int64_t)gridDim.x * 4;
  int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (tile >= a.tiles) return;
  MxUnit m[2][UNITS];
  auto load = [&](int64_t t, MxUnit (&d)[UNITS]) __attribute__((always_inline)) {
    const uint8_t* row = mx_row(a, t < a.tiles ? t : a.tiles - 1, col);   // (past the end: read, not used)
#pragma unroll
    for (int u = 0; u < UNITS; ++u) load_unit(a, row, u, q, d[u]);
  };
  load(tile, m[0]);
  i32x4_t xf[UNITS][8];
#pragma unroll
  for (int u = 0; u < UNITS; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      xf[u][i] = i32x4_t{0, 0, 0, 0};
      if (col < a.N) xf[u][i] = *(const i32x4_t*)(a.X + col * a.ldx + u * 256 + (i / 4) * 128 + 32 * q + 8 * (i % 4));
    }
  for (; tile < a.tiles;) {
    // two turns, so that both buffers have their registers at compile time
    static_for<0, 2>([&](auto d) __attribute__((always_inline)) {
      if (tile >= a.tiles) return;
      load(tile + step, m[d ^ 1]);
      f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          acc = mfma16(xf[u][i], mx_decode8((uint32_t)m[d][u].w[i / 4][i % 4], mx_scale(m[d][u].s[i / 4], q)), acc);
      // loads and stores share one in-order counter: the next tile is awaited before this one's
      // stores are issued, or its wait would be for them as well
      wait_loads();
      store_tile(a, tile, 0, col, q, acc);
      tile += step;
    });
  }
}

// Feature rows in LDS (2 N D bytes), in the order the products take them: chunk k / 8 of all rows,
// then the next chunk, so that a fragment is one conflict-free 16-byte read per lane. Lanes of rows
// from N on read row N - 1: row n of C depends on row n of A alone, and theirs is not stored. A block
// keeps them for all the tiles it takes. KS waves share a tile, each taking every KS-th unit and the
// sums joined through LDS; the next unit's codes are loaded before the present one's products. NT
// tiles of 16 feature rows. Bound by HBM with one row (65536 x 4096 in 28 us, 5.1 TB/s); more rows fall
// off from there (16 rows, 131072 x 4096: 67 us, 4.4 TB/s; 32 rows, 200000 x 768: 31 us, 3.5 TB/s),
// where LDS leaves room for fewer waves and every KiB of codes takes 4 (at 32 rows 8) of fragments from
// LDS. (Weights from HBM at each call; the first and the last take 26 us on weights kept in the last-level cache.)
template <int NT, int KS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_w4_mx_lds(W4Args a) {
  constexpr int GR = WAVES / KS, V = 4 * NT;
  extern __shared__ __attribute__((aligned(16))) i32x4_t xs[];      // [D / 8][N], then the joins
  const int tid = (int)threadIdx.x, wave = tid >> 6, lane = tid & 63, col = lane & 15, q = lane >> 4;
  const int ks = wave % KS, grp = wave / KS;
  const int units = a.units, chunks = 32 * units;
  const int64_t step = (int64_t)gridDim.x * GR, tile00 = (int64_t)blockIdx.x * GR;
  int64_t tile = tile00 + grp;

  MxUnit m[2];
  int64_t lt = tile;
  int lu = ks;
  auto load_next = [&](MxUnit& d) __attribute__((always_inline)) {
    load_unit(a, mx_row(a, lt < a.tiles ? lt : a.tiles - 1, col), a.unit0 + lu, q, d);   // (past the end: read, not used)
    lu += KS;
    if (lu >= units) { lu = ks; lt += step; }
  };
  load_next(m[0]);
  for (int i = tid; i < chunks * a.N; i += 64 * WAVES) {
    const int n = i / chunks, c = i % chunks;              // (consecutive threads read a row)
    xs[c * a.N + n] = *(const i32x4_t*)(a.X + n * a.ldx + 256 * a.unit0 + 8 * c);
  }
  __syncthreads();
  const i32x4_t* x0[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) x0[j] = xs + 4 * q * a.N + (16 * j + col < a.N ? 16 * j + col : a.N - 1);
  float* part = (float*)(xs + chunks * a.N);
  // every wave of a block makes the same number of turns: the joins are barriers
  const int64_t turns = (a.tiles - tile00 + step - 1) / step;
  const int mine = (units - ks + KS - 1) / KS;             // units of this wave per tile (KS <= units)
  f32x4_t acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  int u = ks, buf = 0;
  for (int64_t left = turns * mine; left > 0;) {
    static_for<0, 2>([&](auto d) __attribute__((always_inline)) {
      if (left <= 0) return;
      --left;
      load_next(m[d ^ 1]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const i32x4_t b = mx_decode8((uint32_t)m[d].w[i / 4][i % 4], mx_scale(m[d].s[i / 4], q));
        const int at = (u * 32 + (i / 4) * 16 + i % 4) * a.N;
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j] = mfma16(x0[j][at], b, acc[j]);
      }
      u += KS;
      if (u < units) return;
      u = ks;
      if constexpr (KS == 1) {
#pragma unroll
        for (int j = 0; j < NT; ++j) store_tile(a, tile, 16 * j, col, q, acc[j]);
      } else {
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = acc[i / 4][i % 4];
        join_slices<KS, V>(v, part + (buf * GR + grp) * KS * V * 64, ks, lane, [&](int i, float r) {
          const int n = 16 * (i / 4) + 4 * q + i % 4;
          const int64_t label = tile * 16 + col;
          if (n < a.N && label < a.L) store_result(a, n * a.ldy + label, r);
        });
        buf ^= 1;                                          // one barrier a turn: this half is free again by the next
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      tile += step;
    });
  }
}

// Feature rows that do not fit LDS, where panels do not serve: KS waves share LT tiles, each taking every KS-th
// unit; the rows come from the caches, once per LT tiles, which is more than the weights' own bytes. Sums
// joined through LDS. 16 rows of 16384 features, 32768 labels, BF16 results: 123 us, 2.3 TB/s (FP32
// results, in panels: 91).
template <int NT, int LT, int KS>
__global__ __launch_bounds__(64 * KS) void k_w4_mx_deep(W4Args a) {
  constexpr int V = LT * NT * 4;
  __shared__ float part[KS * V * 64];
  const int ks = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  const int col = lane & 15, q = lane >> 4;
  const int64_t tile0 = (int64_t)blockIdx.x * LT;
  const int units = a.D / 256;
  const uint8_t* row[LT];
#pragma unroll
  for (int t = 0; t < LT; ++t) row[t] = mx_row(a, tile0 + t, col);
  f32x4_t acc[LT][NT];
#pragma unroll
  for (int t = 0; t < LT; ++t)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[t][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  MxUnit m[LT], next[LT];
  int u = ks;
  if (u < units) {
#pragma unroll
    for (int t = 0; t < LT; ++t) load_unit(a, row[t], u, q, m[t]);
  }
  for (; u < units; u += KS) {
    i32x4_t xf[8][NT];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        xf[i][j] = i32x4_t{0, 0, 0, 0};
        if (16 * j + col < a.N)
          xf[i][j] = *(const i32x4_t*)(a.X + (16 * j + col) * a.ldx + u * 256 + (i / 4) * 128 + 32 * q + 8 * (i % 4));
      }
    const int un = u + KS < units ? u + KS : u;
#pragma unroll
    for (int t = 0; t < LT; ++t) load_unit(a, row[t], un, q, next[t]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int t = 0; t < LT; ++t) {
        const float scale = mx_scale(m[t].s[i / 4], q);
        const i32x4_t b = mx_decode8((uint32_t)m[t].w[i / 4][i % 4], scale);
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[t][j] = mfma16(xf[i][j], b, acc[t][j]);
      }
#pragma unroll
    for (int t = 0; t < LT; ++t) m[t] = next[t];
  }
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = acc[i / (4 * NT)][i / 4 % NT][i % 4];
  join_slices<KS, V>(v, part, ks, lane, [&](int i, float s) {
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

// what one lane holds of a unit (128 features) of its label row: 32 codes, and the groups' scales and
// zero points as they lie in memory (128 / G of each)
struct IntUnit { i32x4_t w; i32x2_t s; uint32_t z; };

typedef int i32_a2 __attribute__((aligned(2)));
typedef int i32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef uint16_t u16_a1 __attribute__((aligned(1)));

template <int G>
__device__ __forceinline__ void load_int(const W4Args& a, int64_t label, int u, int q, IntUnit& m) {
  constexpr int GU = 128 / G;
  m.w = i32x4_t{0, 0, 0, 0};
  if (u * 128 + 32 * q < a.D) m.w = *(const i32x4_t*)(a.W + label * (a.D / 2) + u * 64 + 16 * q);   // (whole blocks of 32)
  const int groups = a.D / G, g0 = u * GU;
  const uint16_t* s = a.scales + label * groups + g0;
  const uint8_t* z = a.zeros ? a.zeros + label * groups + g0 : nullptr;
  m.s = i32x2_t{0, 0};
  m.z = 0x08080808u;
  if (g0 + GU <= groups) {
    if constexpr (GU == 4) m.s = *(const i32x2_a2*)s;
    if constexpr (GU == 2) m.s[0] = *(const i32_a2*)s;
    if constexpr (GU == 1) m.s[0] = *s;
    if (z) {
      if constexpr (GU == 4) m.z = *(const u32_a1*)z;
      if constexpr (GU == 2) m.z = *(const u16_a1*)z;
      if constexpr (GU == 1) m.z = *z;
    }
  } else {                                                 // D ends inside the unit: groups past it stay 0
    for (int g = 0; g < groups - g0; ++g) {
      m.s[g >> 1] |= (int)((uint32_t)s[g] << (16 * (g & 1)));
      if (z) m.z = (m.z & ~(255u << (8 * g))) | ((uint32_t)z[g] << (8 * g));
    }
  }
}
// scale and zero point of group g of the unit
__device__ __forceinline__ float int_scale(const IntUnit& m, int g) {
  const uint32_t w = (uint32_t)m.s[g >> 1];
  return u2f(g & 1 ? w & 0xffff0000u : w << 16);
}
__device__ __forceinline__ float int_zero(const IntUnit& m, int g) { return (float)((m.z >> (8 * g)) & 255u); }

// register i of lane (label, q) holds codes 8 i .. of block q -> codes 8 q .. of block i
__device__ __forceinline__ i32x4_t transpose_blocks(i32x4_t w) {
  const auto a = __builtin_amdgcn_permlane32_swap((uint32_t)w[0], (uint32_t)w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap((uint32_t)w[1], (uint32_t)w[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return i32x4_t{(int)c[0], (int)c[1], (int)d[0], (int)d[1]};
}

// A unit's codes against its feature fragments: adds into acc (N <= 4: one result per lane, else four
// per tile of 16 feature rows). frag(j, i): tile j's fragment of chunk i; sum(j, g): the features' own
// sums, N <= 4: of the four blocks of row q, else of group g of rows 4 q .. + 4.
template <int G, int NT, bool FEW, typename X, typename S>
__device__ __forceinline__ void int_unit(const IntUnit& m, float* acc, X&& frag, S&& sum) {
  constexpr int GU = 128 / G;
  const f32x4_t zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (FEW) {
    f32x4_t c = zero4;
#pragma unroll
    for (int i = 0; i < 4; ++i) c = mfma16(frag(0, i), codes8((uint32_t)m.w[i]), c);
    const f32x4_t xs = sum(0, 0);
#pragma unroll
    for (int b = 0; b < 4; ++b)
      acc[0] = __builtin_fmaf(int_scale(m, b * GU / 4), __builtin_fmaf(-int_zero(m, b * GU / 4), xs[b], c[b]), acc[0]);
  } else {
    const i32x4_t t = transpose_blocks(m.w);
    i32x4_t wb[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) wb[b] = codes8((uint32_t)t[b]);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int g = 0; g < GU; ++g) {
        f32x4_t c = zero4;
#pragma unroll
        for (int b = g * (4 / GU); b < (g + 1) * (4 / GU); ++b) c = mfma16(frag(j, b), wb[b], c);
        const f32x4_t xs = sum(j, g);
        const float sc = int_scale(m, g), z = int_zero(m, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[4 * j + i] = __builtin_fmaf(sc, __builtin_fmaf(-z, xs[i], c[i]), acc[4 * j + i]);
      }
  }
}

// Feature rows in LDS as in k_w4_mx_lds ([chunk of 8 features][row], in the decode's order within a
// chunk, a unit of zeros behind the last; N <= 4: lanes outside their block read that at stride 0),
// then the features' sums, [unit][4 q + b] (N <= 4) or [unit][group][row]. KS waves share a tile, each
// taking every KS-th unit, one unit ahead. Groups of 128: one row, 65536 x 4096, in 38 us (3.6 TB/s),
// four in 42, 16 rows, 131072 x 4096, in 104 (2.7 TB/s): below the MXFP4 form's
// 5.1 and 4.4, which has no sums per group and twice the bytes ahead per wave; what bounds this one has
// not been separated.
template <int G, int NT, bool FEW, int KS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_w4_int_lds(W4Args a) {
  constexpr int GR = WAVES / KS, SB = FEW ? 4 : 128 / G, V = FEW ? 1 : 4 * NT, SR = FEW ? 4 : 16 * NT;
  extern __shared__ __attribute__((aligned(16))) i32x4_t xs[];
  const int tid = (int)threadIdx.x, wave = tid >> 6, lane = tid & 63, col = lane & 15, q = lane >> 4;
  const int ks = wave % KS, grp = wave / KS, N = a.N;
  const int units = a.units;
  const int64_t step = (int64_t)gridDim.x * GR, tile00 = (int64_t)blockIdx.x * GR;
  int64_t tile = tile00 + grp;
  float* sums = (float*)(xs + (units + 1) * 16 * N);
  float* part = sums + (units + 1) * SB * SR;

  IntUnit m[2];
  int64_t lt = tile;
  int lu = ks;
  auto load_next = [&](IntUnit& d) __attribute__((always_inline)) {
    int64_t label = (lt < a.tiles ? lt : a.tiles - 1) * 16 + col;    // (past the end: read, not used)
    if (label >= a.L) label = a.L - 1;
    load_int<G>(a, label, a.unit0 + lu, q, d);
    lu += KS;
    if (lu >= units) { lu = ks; lt += step; }
  };
  load_next(m[0]);
  // thread by (row, block or group): its 16-byte chunks, and its sum in the order of the features
  for (int j = tid; j < (units + 1) * SB * N; j += 64 * WAVES) {
    const int n = j / ((units + 1) * SB), ug = j % ((units + 1) * SB), u = ug / SB, g = ug % SB;
    float sum = 0.0f;
    for (int c = ug * (16 / SB); c < (ug + 1) * (16 / SB); ++c) {
      i32x4_t v = {0, 0, 0, 0};
      if (u < units && 128 * a.unit0 + 8 * c < a.D) v = *(const i32x4_t*)(a.X + n * a.ldx + 128 * a.unit0 + 8 * c);
      float f[8];
      ElemBF16::widen(v, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += f[e];
      xs[c * N + n] = even_odd(v);
    }
    sums[FEW ? u * 16 + 4 * n + g : (u * SB + g) * SR + n] = sum;
  }
  __syncthreads();
  // lane's place in A: row col, which is feature row 16 j + col, or col / 4 in block col % 4
  const bool own = !FEW || (col & 3) == q;
  int xrow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int n = FEW ? col >> 2 : 16 * j + col;           // (rows past N: row N - 1, not stored)
    xrow[j] = (FEW ? 4 * q : q) * N + (n < N ? n : N - 1) + (own ? 0 : units * 16 * N);
  }
  const int ustride = own ? 16 * N : 0, cstride = FEW ? N : 4 * N;
  const int64_t turns = (a.tiles - tile00 + step - 1) / step;
  const int mine = (units - ks + KS - 1) / KS;             // (KS <= units)
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.0f;
  int u = ks, buf = 0;
  for (int64_t left = turns * mine; left > 0;) {
    static_for<0, 2>([&](auto d) __attribute__((always_inline)) {
      if (left <= 0) return;
      --left;
      load_next(m[d ^ 1]);
      int_unit<G, NT, FEW>(
          m[d], acc, [&](int j, int i) __attribute__((always_inline)) { return xs[xrow[j] + u * ustride + i * cstride]; },
          [&](int j, int g) __attribute__((always_inline)) {
            return *(const f32x4_t*)&sums[FEW ? u * 16 + 4 * q : (u * SB + g) * SR + 16 * j + 4 * q];
          });
      u += KS;
      if (u < units) return;
      u = ks;
      join_slices<KS, V>(acc, part + (buf * GR + grp) * KS * V * 64, ks, lane, [&](int j, float r) {
        const int n = FEW ? q : 16 * (j / 4) + 4 * q + j % 4;
        const int64_t label = tile * 16 + col;
        if (tile < a.tiles && n < N && label < a.L) store_result(a, n * a.ldy + label, r);
      });
      if constexpr (WAVES == 16) __syncthreads();          // (one buffer: its readers are done)
      else buf ^= 1;                                       // (two: free again by the turn after next)
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = 0.0f;
      tile += step;
    });
  }
}

// Feature rows that do not fit LDS, where panels do not serve: the rows from the caches, their sums as
// products against ones. 24 rows of 8192 features, 32768 labels, BF16 results, in 145 us (1.0 TB/s): the
// rows are read once per tile, six times the weights' bytes. With FP32 results, in panels, 102.
template <int G, int NT, bool FEW, int KS>
__global__ __launch_bounds__(64 * KS) void k_w4_int_deep(W4Args a) {
  constexpr int V = FEW ? 1 : 4 * NT, GU = 128 / G;
  __shared__ float part[KS * V * 64];
  const int ks = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  const int col = lane & 15, q = lane >> 4;
  const int64_t tile = a.tile0 + blockIdx.x;
  int64_t label = tile * 16 + col;
  if (label >= a.L) label = a.L - 1;
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.0f;
  const int units = (a.D + 127) / 128;
  const i32x4_t one = {0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80};
  for (int u = ks; u < units; u += KS) {
    IntUnit m;
    load_int<G>(a, label, u, q, m);
    i32x4_t xf[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = FEW ? col >> 2 : 16 * j + col, k = u * 128 + (FEW ? 32 * q + 8 * i : 32 * i + 8 * q);
        xf[j][i] = i32x4_t{0, 0, 0, 0};
        if (k < a.D && n < a.N && (!FEW || (col & 3) == q)) xf[j][i] = even_odd(*(const i32x4_t*)(a.X + n * a.ldx + k));
      }
    int_unit<G, NT, FEW>(
        m, acc, [&](int j, int i) __attribute__((always_inline)) { return xf[j][i]; },
        [&](int j, int g) __attribute__((always_inline)) {
          f32x4_t c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = FEW ? 0 : g * (4 / GU); i < (FEW ? 4 : (g + 1) * (4 / GU)); ++i) c = mfma16(xf[j][i], one, c);
          return c;
        });
  }
  join_slices<KS, V>(acc, part, ks, lane, [&](int j, float s) {
    const int n = FEW ? q : 16 * (j / 4) + 4 * q + j % 4;
    const int64_t lab = tile * 16 + col;
    if (n < a.N && lab < a.L) store_result(a, n * a.ldy + lab, s);
  });
}

// ---- launchers -------------------------------------------------------------------------------------
constexpr size_t W4_LDS = 160 << 10;                       // per CU and per block

// Lets a kernel take all of it. The limit belongs to the process, so it is the same for every call: one
// set to a call's own size could be lowered by another host thread between this and the launch.
static bool raise_lds_limit(const void* kernel, size_t lds) {
  return lds <= (64 << 10) || hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)W4_LDS) == hipSuccess;
}

template <int UNITS>
static int go_regs(const W4Args& a, hipStream_t st) {
  const int64_t want = (a.tiles + 3) / 4, cap = 2 * (int64_t)device_cus();   // 2 waves per SIMD at 200-240 registers
  hipLaunchKernelGGL(k_w4_mx_regs<UNITS>, dim3((unsigned)(want < cap ? want : cap)), dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
}
static size_t mx_lds_bytes(const W4Args& a, int units, int NT, int KS, int WAVES) {
  return (size_t)units * 512 * a.N + (KS > 1 ? (size_t)2 * WAVES * NT * 1024 : 0);
}
template <int NT, int KS, int WAVES>
static int go_lds(const W4Args& a, hipStream_t st) {
  constexpr int GR = WAVES / KS;
  const size_t lds = mx_lds_bytes(a, a.units, NT, KS, WAVES);
  int per_cu = (int)(W4_LDS / lds);
  if (per_cu > 16 / WAVES) per_cu = 16 / WAVES;            // 4 waves per SIMD
  if (per_cu < 1) per_cu = 1;
  const int64_t want = (a.tiles + GR - 1) / GR, cap = (int64_t)device_cus() * per_cu;
  if (!raise_lds_limit((const void*)k_w4_mx_lds<NT, KS, WAVES>, lds)) return ELMO_EHIP_;
  hipLaunchKernelGGL((k_w4_mx_lds<NT, KS, WAVES>), dim3((unsigned)(want < cap ? want : cap)), dim3(64 * WAVES), lds, st, a);
  return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
}
template <int NT, int LT, int KS>
static int go_deep(const W4Args& a, hipStream_t st) {      // (2^32 threads are 2^28 labels here, over 300 GB of weights)
  hipLaunchKernelGGL((k_w4_mx_deep<NT, LT, KS>), dim3((unsigned)((a.tiles + LT - 1) / LT)), dim3(64 * KS), 0, st, a);
  return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
}
// Runs `go` on panels of `units` units that fit LDS with 8 waves each (lds(n): bytes for n units), as
// equal as they come, adding the results of all but the first. False, and nothing run, where that takes
// several panels and either their sums would have to round (16-bit results) or there are too few tiles
// to be worth staging the rows of each: 24 rows of 4864 features against 113635 integer labels take 142
// us in panels and 300 with the rows from the caches, 12 rows of 8192 against 4096 labels 25 and 17.
template <typename B, typename G>
static bool in_panels(const W4Args& a, int units, B&& lds, G&& go, int& rc) {
  int most = units;
  while (most > 1 && lds(most) > W4_LDS) --most;
  const int panels = (units + most - 1) / most, per = (units + panels - 1) / panels;
  if (panels > 1 && (a.ytype != T_F32_ || a.tiles <= 4 * device_cus())) return false;
  rc = ELMO_OK_;
  for (int u = 0; u < units && rc == ELMO_OK_; u += per) {
    W4Args p = a;
    p.unit0 = u;
    p.units = units - u < per ? units - u : per;
    p.add = u > 0;
    rc = go(p);
  }
  return true;
}

template <int NT>
static int pick_mx(const W4Args& a, hipStream_t st) {
  int rc;
  const bool done = in_panels(
      a, a.D / 256, [&](int n) { return mx_lds_bytes(a, n, NT, n < 8 ? 1 : 8, 8); },
      [&](const W4Args& p) {
        if (p.units < 8) {
          // (16 rows of up to 7 units always leave room for two blocks)
          if constexpr (NT > 1) {
            if (2 * mx_lds_bytes(p, p.units, NT, 1, 4) > W4_LDS) return go_lds<NT, 1, 16>(p, st);
          }
          return go_lds<NT, 1, 4>(p, st);
        }
        // where only one block fits a CU, 16 waves of it hide more latency than 8, unless there are too
        // few tiles to give both groups a share
        if (2 * mx_lds_bytes(p, p.units, NT, 8, 8) > W4_LDS && p.tiles >= 4 * device_cus() &&
            mx_lds_bytes(p, p.units, NT, 8, 16) <= W4_LDS)
          return go_lds<NT, 8, 16>(p, st);
        return go_lds<NT, 8, 8>(p, st);
      },
      rc);
  return done ? rc : go_deep<NT, 2, 8>(a, st);
}

template <int G, int NT, bool FEW, int KS, int WAVES>
static size_t int_lds_bytes(const W4Args& a, int units) {
  const size_t sums = FEW ? 64 : (128 / G) * NT * 64;
  return ((size_t)units + 1) * (256 * a.N + sums) + (KS > 1 ? (size_t)(WAVES == 16 ? 1 : 2) * WAVES * (FEW ? 1 : 4 * NT) * 256 : 0);
}
template <int G, int NT, bool FEW, int KS, int WAVES>
static int go_int(const W4Args& a, hipStream_t st) {
  constexpr int GR = WAVES / KS;
  const size_t lds = int_lds_bytes<G, NT, FEW, KS, WAVES>(a, a.units);
  int per_cu = (int)(W4_LDS / lds);
  if (per_cu > 24 / WAVES) per_cu = 24 / WAVES;            // 6 waves per SIMD (65536 x 4096, one row: 36.5 us; at 4: 41.7)
  if (per_cu < 1) per_cu = 1;
  const int64_t want = (a.tiles + GR - 1) / GR, cap = (int64_t)device_cus() * per_cu;
  if (!raise_lds_limit((const void*)k_w4_int_lds<G, NT, FEW, KS, WAVES>, lds)) return ELMO_EHIP_;
  hipLaunchKernelGGL((k_w4_int_lds<G, NT, FEW, KS, WAVES>), dim3((unsigned)(want < cap ? want : cap)), dim3(64 * WAVES), lds, st, a);
  return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
}
template <int G, int NT, bool FEW>
static int pick_int(const W4Args& a, hipStream_t st) {
  int rc;
  const bool done = in_panels(
      a, (a.D + 127) / 128,
      [&](int n) { return n < 8 ? int_lds_bytes<G, NT, FEW, 1, 4>(a, n) : int_lds_bytes<G, NT, FEW, 8, 8>(a, n); },
      [&](const W4Args& p) {
        if (p.units < 8) return go_int<G, NT, FEW, 1, 4>(p, st);
        if (2 * int_lds_bytes<G, NT, FEW, 8, 8>(p, p.units) > W4_LDS && p.tiles >= 4 * device_cus() &&
            int_lds_bytes<G, NT, FEW, 8, 16>(p, p.units) <= W4_LDS)
          return go_int<G, NT, FEW, 8, 16>(p, st);
        return go_int<G, NT, FEW, 8, 8>(p, st);
      },
      rc);
  if (done) return rc;
  // a launch holds fewer than 2^32 threads: runs of at most 2^22 tiles (2^26 labels)
  constexpr int64_t MOST = int64_t(1) << 22;
  W4Args p = a;
  for (; p.tile0 < a.tiles; p.tile0 += MOST) {
    const int64_t left = a.tiles - p.tile0;
    hipLaunchKernelGGL((k_w4_int_deep<G, NT, FEW, 8>), dim3((unsigned)(left < MOST ? left : MOST)), dim3(512), 0, st, p);
    if (hipGetLastError() != hipSuccess) return ELMO_EHIP_;
  }
  return ELMO_OK_;
}
template <int G>
static int pick_rows(const W4Args& a, hipStream_t st) {
  if (a.N <= 4) return pick_int<G, 1, true>(a, st);
  if (a.N <= 16) return pick_int<G, 1, false>(a, st);
  return pick_int<G, 2, false>(a, st);
}

static int pick_format(const W4Args& a, int wdtype, hipStream_t st) {
  if (wdtype == W_MXFP4_) {
    if (a.N > 16) return pick_mx<2>(a, st);
    switch (a.D / 256) {
      case 1: return go_regs<1>(a, st);
      case 2: return go_regs<2>(a, st);
      case 3: return go_regs<3>(a, st);
      case 4: return go_regs<4>(a, st);
      default: return pick_mx<1>(a, st);
    }
  }
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
