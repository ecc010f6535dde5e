// Log probabilities of given labels straight from features and weights, and the gradient: softmax cross
// entropy of a linear head whose logits are never kept.
//
// Forward: Z = X W^T tile by tile (256 labels x 256 rows, or less); each wave reduces its labels to a maximum and a
// sum of e^(z - max) per row (8 bytes for 128 logits) and picks the given labels' logits out. 4,096 x 131,072 x 768:
// 720 us, 1,145 TFLOP/s (the library's product alone 700). One row of 131,072 x 768: 40 us, 5.0 TB/s of weights. A
// second kernel joins the parts of a row.
//
// Backward, a piece of the vocabulary at a time: the piece's logits again, as G = c_n p + (given labels'
// gradients) in 16 bits in the workspace, then dX += G W and dW = G^T X in one launch or two. G is the one
// rounding below 32 bits: half a unit of its type per element, of its own size (c p of a label that was
// not given, c p + g of one that was, added before it is rounded, so that a label of probability near 1
// keeps the digits of 1 - p). G is scaled by the largest given gradient: the constant gradient 1 / N of
// a mean then is exactly 1, and in FP16 a power of two more keeps p down to 2^-38. Up to 128 rows G
// is held as the sum of two 16-bit numbers, in rows n and N + n: few rows do not average their roundings, and
// memory bounds such products. Above that it is so where a result is FP32, whose own rounding does not hide that of
// G; the products of that result take twice the operations. 4,096 x 131,072 x 768: 2.5 ms, 980 TFLOP/s over the three
// products, with BF16 results (off by 1.9e-3 and 1.7e-3 of their norms, 1.7e-3 and 1.5e-3 with an exact G); 3.4 ms with
// dW, 3.7 ms with dX in FP32 (2.6 and 2.5 from one number; off by 1.5e-6 for 9.4e-4).
#include <cfloat>

#include "tile_shapes.hpp"

namespace elmo {

constexpr float L2E = 1.44269502162933349609375f;          // FP32(log2 e)
// e^(z - m) is formed as 2^(z L2E - b), b = FP32(m L2E), and what b's rounding leaves out as a factor, while |b| is below
// FAR: the factor then is at most 2^(1/2). From 2^31 on it would leave binary32's range. Rows beyond FAR take z - m first
// (one more operation a logit, of the waves that have such a row), rows below it keep their bits next to them.
constexpr float FAR = 16777216.0f;
constexpr int COEF_THREADS = 1024;
constexpr int GROUP = 8;                                   // label tiles that are taken together over the rows

// ---- logits ----------------------------------------------------------------------------------------
struct LogitTiles {
  const char* X; const char* W;
  int64_t ldx, ldw;                                        // bytes
  int64_t N, v0, v1;                                       // rows; labels of the piece
  int stages, row_tiles, label_tiles;
  __device__ __forceinline__ void place(int u, int& lt, int& nt) const {
    const int per = GROUP * row_tiles, g = u / per, r = u % per;
    const int wide = label_tiles - g * GROUP < GROUP ? label_tiles - g * GROUP : GROUP;
    nt = r / wide;
    lt = g * GROUP + r % wide;
  }
  template <class S>
  __device__ __forceinline__ TileUnit unit(int u) const {
    int lt, nt;
    place(u, lt, nt);
    const int64_t l = v0 + (int64_t)lt * S::M, n = (int64_t)nt * S::N;
    return {{W + l * ldw, ldw, v1 - l, 0}, {X + n * ldx, ldx, N - n, 0}, stages};
  }
};

// where a wave's ROWS labels from l0 on have a given label: 32 i + 8 (r / 4) + r % 4 of the lane that
// holds it, else negative
template <int ROWS>
__device__ __forceinline__ int given_place(int id, int64_t l0, int64_t v1, int half) {
  const int64_t at = (int64_t)id - l0;
  if (at < 0 || at >= ROWS || id >= v1 || (((int)at >> 2) & 1) != half) return -1;
  return (int)at - 4 * half;
}

// Whether any of the wave's rows from n0 on has a given label among the `labels` from l0 on. All their ids in lane
// order, so that the loads are on their way together; a tile without one (most, over many labels) is done with
// it. (8 labels a row looked up row by row took a tenth of the time of 1,001 x 670,000 x 768.)
template <int ROWS>
__device__ __forceinline__ bool any_given(const int32_t* ids, int64_t n0, int64_t N, int M, int64_t l0, int labels, int lane) {
  const int64_t rows = N - n0 < ROWS ? N - n0 : ROWS;
  const int count = rows > 0 ? (int)rows * M : 0;
  const int32_t* p = ids + n0 * M;
  bool any = false;
#pragma unroll 8
  for (int k = lane; k < count; k += 64) {
    const int64_t at = (int64_t)p[k] - l0;
    any |= at >= 0 && at < labels;
  }
  return __any(any);
}

struct StatArgs {
  LogitTiles t;
  const int32_t* ids; int M;
  float2* part;                                            // [parts of 32 MF labels][N]: maximum, sum
  float* given;                                            // [N][M]: logits of the given labels
};

template <class S>
struct StatJob : StatArgs {
  static constexpr int STORES = S::NF;
  __device__ __forceinline__ TileUnit unit(int u) const { return t.unit<S>(u); }
  __device__ __forceinline__ bool finish(int u, f32x16_t (&acc)[S::MF][S::NF], int wm, int wn, int lane, char* lds) const {
    int lt, nt;
    t.place(u, lt, nt);
    const int64_t l0 = (int64_t)lt * S::M + S::WM_ROWS * wm, n0 = (int64_t)nt * S::N + S::WN_ROWS * wn;
    const int half = lane >> 5;
    const int64_t left = t.v1 - l0;                        // (wave-uniform)
    const bool given_here = any_given<S::WN_ROWS>(ids, n0, t.N, M, l0, S::WM_ROWS, lane);
    int64_t n[S::NF];
#pragma unroll
    for (int j = 0; j < S::NF; ++j) n[j] = n0 + 32 * j + (lane & 31);
    if (left < S::WM_ROWS) {
      const int mine = (int)(left < -128 ? -128 : left) - 4 * half;
#pragma unroll
      for (int i = 0; i < S::MF; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (32 * i + 8 * (r / 4) + r % 4 >= mine) 
#pragma unroll
            for (int j = 0; j < S::NF; ++j) acc[i][j][r] = -__builtin_inff();
    }
#pragma unroll
    for (int j = 0; j < S::NF; ++j) {
      float top = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < S::MF; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, acc[i][j][r]);
      top = fmaxf(top, __shfl_xor(top, 32));
      for (int g = 0; given_here && g < M; ++g) {
        const int id = n[j] < t.N ? ids[n[j] * M + g] : -1;
        const int at = given_place<S::WM_ROWS>(id, l0, t.v1, half);
        const bool hit = at >= 0;
        if (__any(hit)) {
          float z = 0.0f;
#pragma unroll
          for (int i = 0; i < S::MF; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              if (at == 32 * i + 8 * (r / 4) + r % 4) z = acc[i][j][r];
          if (hit) given[n[j] * M + g] = z;
        }
      }
      float ref = top == -__builtin_inff() ? 0.0f : top;
      const bool far = fabsf(ref) * L2E >= FAR && fabsf(ref) < __builtin_inff();
      if (__any(far)) {
        const float off = far ? ref : 0.0f;
        if (far) ref = 0.0f;
#pragma unroll
        for (int i = 0; i < S::MF; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][j][r] -= off;
      }
      // e^(z - top) as 2^(z L2E - b), b = FP32(top L2E): what b's rounding leaves out is a factor of the sum
      const float b = ref * L2E, rest = __builtin_fmaf(ref, L2E, -b);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < S::MF; ++i) {
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) s += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][r], L2E, -b));
        sum += s;
      }
      sum += __shfl_xor(sum, 32);
      sum *= __builtin_amdgcn_exp2f(-rest);
      if (half == 0 && n[j] < t.N) part[((int64_t)lt * 2 + wm) * t.N + n[j]] = make_float2(top, sum);
    }
    return n0 + S::WN_ROWS <= t.N;
  }
};

template <class Mul, class S>
__global__ __launch_bounds__(S::THREADS, S::WAVES) void k_lin_stats(StatArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[S::lds(false)];
  StatJob<S> job;
  (StatArgs&)job = a;
  const UnitRange r = xcd_units(a.t.label_tiles * a.t.row_tiles);
  tile_stream<Mul, false, false, S>(job, r.first, r.step, r.end, lds);
}

// The parts of `wide` rows from n0 on (a power of two up to 16) joined by a block: 1024 / wide runs of parts a row, then the runs in
// the order of a tree.
__global__ __launch_bounds__(1024) void k_lin_join(const float2* part, int64_t parts, int64_t n0, int64_t N, int64_t V, int wide, const int32_t* ids,
                                                   int M, const float* given, float* logp, float* row_max, float* log_sum) {
  __shared__ float2 joined[1024];
  const int tid = (int)threadIdx.x, x = tid & (wide - 1), y = tid / wide, runs = 1024 / wide;
  const int64_t n = n0 + (int64_t)blockIdx.x * wide + x;
  float top = -__builtin_inff(), sum = 0.0f;
  auto add = [&](float m, float s) {
    const float hi = fmaxf(top, m);
    const float ref = hi == -__builtin_inff() ? 0.0f : hi;
    sum = sum * __builtin_amdgcn_exp2f((top - ref) * L2E) + s * __builtin_amdgcn_exp2f((m - ref) * L2E);
    top = hi;
  };
  if (n < N) {
#pragma unroll 8
    for (int64_t p = y; p < parts; p += runs) {
      const float2 v = part[p * N + n];
      add(v.x, v.y);
    }
  }
  joined[tid] = make_float2(top, sum);
  for (int k = 512; k >= wide; k >>= 1) {
    __syncthreads();
    if (tid < k) {
      add(joined[tid + k].x, joined[tid + k].y);
      joined[tid] = make_float2(top, sum);
    }
  }
  __syncthreads();
  if (n >= N) return;
  top = joined[x].x;
  sum = joined[x].y;
  const bool empty = top == -__builtin_inff() && sum == 0.0f;
  const float logs = empty ? 0.0f : logf(sum);
  if (y == 0) {
    row_max[n] = top;
    log_sum[n] = logs;
  }
  for (int g = y; g < M; g += runs) {
    const int id = ids[n * M + g];
    float v = 0.0f;
    if (id >= V) v = __builtin_nanf("");
    else if (id >= 0) v = empty ? -__builtin_inff() : (given[n * M + g] - top) - logs;
    logp[n * M + g] = v;
  }
}

// ---- gradient --------------------------------------------------------------------------------------
struct CoefArgs {
  int64_t N, V; int M;
  const int32_t* ids;
  const float *row_max, *log_sum, *dlogp, *dlse;
  float2* most; int parts;                                 // maxima of runs of rows, if taken by themselves
  float2* coef;                                            // [N]: b, c 2^(what b's rounding left out), scaled; |b| >= FAR: no such factor
  float* up;                                               // [N][M]: the given labels' gradients, scaled
  float* inv;                                              // 1 / scale
  int f16;
};

// the largest given gradient of a row (of finite ones), and the bound of |G| in it: FLT_MAX where that is larger (by a factor
// of at most 1 + 2 ELMO_MAX_GIVEN < 2^8), 0 for a row with a NaN or an infinity
__device__ __forceinline__ float2 row_bound(const CoefArgs& a, int64_t n) {
  float most = 0.0f, all = a.dlse ? fabsf(a.dlse[n]) : 0.0f;
  bool finite = all < __builtin_inff();
  for (int g = 0; g < a.M; ++g) {
    const int id = a.ids[n * a.M + g];                     // (both loads are on their way together)
    const float d = fabsf(a.dlogp[n * a.M + g]);
    if (id >= 0 && d < __builtin_inff()) most = fmaxf(most, d);
    if (id >= 0) {
      all += 2.0f * d;
      finite = finite && d < __builtin_inff();
    }
  }
  return make_float2(most, finite ? fminf(all, FLT_MAX) : 0.0f);
}
__device__ __forceinline__ float2 block_max(float2 v, float2* s) {
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) {
    v.x = fmaxf(v.x, __shfl_xor(v.x, k));
    v.y = fmaxf(v.y, __shfl_xor(v.y, k));
  }
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < COEF_THREADS / 64; ++w) {
    v.x = fmaxf(v.x, s[w].x);
    v.y = fmaxf(v.y, s[w].y);
  }
  return v;
}

__global__ __launch_bounds__(COEF_THREADS) void k_lin_bound(CoefArgs a) {
  __shared__ float2 s[COEF_THREADS / 64];
  float2 v = make_float2(0.0f, 0.0f);
  for (int64_t n = blockIdx.x * (int64_t)COEF_THREADS + threadIdx.x; n < a.N; n += (int64_t)gridDim.x * COEF_THREADS) {
    const float2 r = row_bound(a, n);
    v.x = fmaxf(v.x, r.x);
    v.y = fmaxf(v.y, r.y);
  }
  v = block_max(v, s);
  if (threadIdx.x == 0) a.most[blockIdx.x] = v;
}

__global__ __launch_bounds__(COEF_THREADS) void k_lin_coef(CoefArgs a) {
  __shared__ float2 s[COEF_THREADS / 64];
  float2 v = make_float2(0.0f, 0.0f);
  if (a.parts > 0) {
    for (int i = (int)threadIdx.x; i < a.parts; i += COEF_THREADS) {
      v.x = fmaxf(v.x, a.most[i].x);
      v.y = fmaxf(v.y, a.most[i].y);
    }
  } else {
#pragma unroll 4
    for (int64_t n = threadIdx.x; n < a.N; n += COEF_THREADS) {
      const float2 r = row_bound(a, n);
      v.x = fmaxf(v.x, r.x);
      v.y = fmaxf(v.y, r.y);
    }
  }
  v = block_max(v, s);
  // unit: what becomes 1 (the largest given gradient, unless the bound is more than 2^60 times that; or else the
  // bound); FP16: times the power of two that brings the bound into [2^14, 2^15), as far as its inverse is finite
  float unit = v.x > 0.0f ? fmaxf(v.x, 0x1p-60f * v.y) : v.y;
  unit = fminf(fmaxf(unit, 1e-30f), 1e30f);
  if (a.f16) {
    const float ratio = fmaxf(v.y / unit, 1e-30f);
    unit = fmaxf(ldexpf(unit, __builtin_amdgcn_frexp_expf(ratio) - (v.y == FLT_MAX ? 15 - 8 : 15)), 1.17549435e-38f);   // (2^-126)
  }
  const float scale = 1.0f / unit;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.inv = unit;
  const int64_t n = blockIdx.x * (int64_t)COEF_THREADS + threadIdx.x;
  if (n >= a.N) return;
  const double lse = (double)a.row_max[n] + (double)a.log_sum[n];
  const bool empty = lse == -__builtin_inf();
  float c = a.dlse ? a.dlse[n] : 0.0f, scaled = c * scale;   // (scaled: for a sum beyond binary32's range)
  for (int g = 0; g < a.M; ++g) {
    const int id = a.ids[n * a.M + g];
    float d = 0.0f;
    if (id >= 0) d = a.dlogp[n * a.M + g];
    if (id >= a.V) c = scaled = __builtin_nanf("");
    c -= d;
    scaled -= d * scale;
    a.up[n * a.M + g] = empty ? 0.0f : d * scale;
  }
  if (fabsf(c) < __builtin_inff()) scaled = c * scale;
  // p = 2^(z L2E - lse L2E): exact for z = lse, where 1 - p needs it
  const double bd = empty ? 0.0 : lse * (double)L2E;
  const float b = (float)bd;
  const float rest = fabsf(b) >= FAR ? 0.0f : (float)(bd - (double)b);
  a.coef[n] = make_float2(b, empty ? 0.0f : scaled * __builtin_amdgcn_exp2f(-rest));
}

template <class Mul>
__device__ __forceinline__ int pack16(float lo, float hi) {
  if constexpr (std::is_same_v<Mul, MulF16>) {
    typedef _Float16 f16x2_v __attribute__((ext_vector_type(2)));
    typedef float f32x2_v __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(int, __builtin_convertvector((f32x2_v){lo, hi}, f16x2_v));
  } else {
    return (int)pack_bf16x2(lo, hi);
  }
}

// what rounding to 16 bits leaves of two values
template <class Mul>
__device__ __forceinline__ int rest16(float lo, float hi) {
  const int w = pack16<Mul>(lo, hi);
  float f[8];
  std::conditional_t<std::is_same_v<Mul, MulF16>, ElemF16, ElemBF16>::widen(i32x4_t{w, 0, 0, 0}, f);
  return pack16<Mul>(lo - f[0], hi - f[1]);
}

struct GradArgs {
  LogitTiles t;
  int planes;                                              // 2: G as two numbers
  const int32_t* ids; int M;
  const float2* coef; const float* up;
  const float *row_max, *log_sum;                          // of rows beyond FAR
  char* G; int64_t ldg;                                    // [N] rows of the piece's labels; bytes
};

template <class Mul, class S>
struct GradJob : GradArgs {
  static constexpr int STORES = S::NF * S::PIECES / 2;
  __device__ __forceinline__ TileUnit unit(int u) const { return t.unit<S>(u); }
  __device__ __forceinline__ bool finish(int u, f32x16_t (&acc)[S::MF][S::NF], int wm, int wn, int lane, char* lds) const {
    int lt, nt;
    t.place(u, lt, nt);
    const int64_t col0 = (int64_t)lt * S::M + S::WM_ROWS * wm, n0 = (int64_t)nt * S::N + S::WN_ROWS * wn;
    const int half = lane >> 5;
    const int64_t l0 = t.v0 + col0, left = t.v1 - l0;      // (wave-uniform)
    const bool given_here = any_given<S::WN_ROWS>(ids, n0, t.N, M, l0, S::WM_ROWS, lane);
    int64_t n[S::NF];
    float2 cf[S::NF];
#pragma unroll
    for (int j = 0; j < S::NF; ++j) {
      n[j] = n0 + 32 * j + (lane & 31);
      const bool in = n[j] < t.N;
      cf[j] = in ? coef[n[j]] : make_float2(0.0f, 0.0f);
    }
#pragma unroll
    for (int j = 0; j < S::NF; ++j) {
      const bool far = fabsf(cf[j].x) >= FAR;
      if (__any(far)) {                                    // (z - row_max) L2E - log_sum L2E
        const float off = far ? row_max[n[j]] : 0.0f;
        if (far) cf[j].x = log_sum[n[j]] * L2E;
#pragma unroll
        for (int i = 0; i < S::MF; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][j][r] -= off;
      }
#pragma unroll
      for (int i = 0; i < S::MF; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          acc[i][j][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][r], L2E, -cf[j].x)) * cf[j].y;
      for (int g = 0; given_here && g < M; ++g) {
        const int id = n[j] < t.N ? ids[n[j] * M + g] : -1;
        const int at = given_place<S::WM_ROWS>(id, l0, t.v1, half);
        const bool hit = at >= 0;
        if (__any(hit)) {
          const float d = hit ? up[n[j] * M + g] : 0.0f;
#pragma unroll
          for (int i = 0; i < S::MF; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              acc[i][j][r] += at == 32 * i + 8 * (r / 4) + r % 4 ? d : 0.0f;
        }
      }
    }
    if (left < S::WM_ROWS) {                                      // labels past the last: no share in dX
      const int mine = (int)(left < -128 ? -128 : left) - 4 * half;
#pragma unroll
      for (int i = 0; i < S::MF; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (32 * i + 8 * (r / 4) + r % 4 >= mine) 
#pragma unroll
            for (int j = 0; j < S::NF; ++j) acc[i][j][r] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < S::NF; ++j) {
      i32x4_t v[2 * S::MF];
      pieces16<S::MF>(acc, j, v, [](float lo, float hi) { return pack16<Mul>(lo, hi); });
      const int64_t r0 = n0 + 32 * j;
      put_rows<S::PIECES>(lds, lane, v, [&](int row, int c, i32x4_t x) {
        if (r0 + row < t.N) *(i32x4_t*)(G + (r0 + row) * ldg + 2 * col0 + 16 * c) = x;
      });
      if (planes == 1) continue;
      pieces16<S::MF>(acc, j, v, [](float lo, float hi) { return rest16<Mul>(lo, hi); });
      put_rows<S::PIECES>(lds, lane, v, [&](int row, int c, i32x4_t x) {
        if (r0 + row < t.N) *(i32x4_t*)(G + (t.N + r0 + row) * ldg + 2 * col0 + 16 * c) = x;
      });
    }
    return n0 + S::WN_ROWS <= t.N;
  }
};

template <class Mul, class S>
__global__ __launch_bounds__(S::THREADS, S::WAVES) void k_lin_grad_logits(GradArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[S::lds(true)];
  GradJob<Mul, S> job;
  (GradArgs&)job = a;
  const UnitRange r = xcd_units(a.t.label_tiles * a.t.row_tiles);
  tile_stream<Mul, false, false, S>(job, r.first, r.step, r.end, lds);
}

// dW = G^T X: rows of the result are labels (n of the tile), its columns features (m)
struct OutArgs { void* out; int64_t ld; int type; int accumulate; };   // ld in elements
struct ProductArgs {
  const char* X; int64_t ldx;
  const char* W; int64_t ldw;
  const char* G; int64_t ldg;
  int64_t N, v0, v1, cols;                                 // cols: the piece's labels, a multiple of 256
  int w_planes, x_planes;                                  // 2: with both numbers of G, of which the second starts at row N
  int D, d_tiles, row_tiles;
  const float* inv;
  // dW: the tokens in w_slots runs of w_per; one run goes to the result, several to `wpart`
  int w_units, w_slots; int64_t w_per;
  float* wpart; OutArgs dW;
  // dX: the piece's labels in x_slots runs of x_per, each added to its partial sum; or (xpart NULL) one run over all
  // labels, which goes to the result
  int x_units, x_slots, x_heavy, x_light, first; int64_t x_per;
  float* xpart; OutArgs dX;
};

__device__ __forceinline__ void store4(const OutArgs& o, int64_t row, int64_t col, f32x4_t v) {
  if (o.type == T_F32_) {
    f32x4_t* p = (f32x4_t*)((float*)o.out + row * o.ld + col);
    *p = o.accumulate ? *p + v : v;
  } else {
    uint16_t* p = (uint16_t*)o.out + row * o.ld + col;
    i32x2_t w = *(const i32x2_t*)p;
    if (o.type == T_BF16_) {
      if (o.accumulate) v += f32x4_t{bf16_to_f32(w[0] & 0xffff), bf16_to_f32((uint32_t)w[0] >> 16), bf16_to_f32(w[1] & 0xffff), bf16_to_f32((uint32_t)w[1] >> 16)};
      w = i32x2_t{pack16<MulBF16>(v[0], v[1]), pack16<MulBF16>(v[2], v[3])};
    } else {
      if (o.accumulate)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += (float)__builtin_bit_cast(_Float16, (uint16_t)((uint32_t)w[i / 2] >> 16 * (i % 2)));
      w = i32x2_t{pack16<MulF16>(v[0], v[1]), pack16<MulF16>(v[2], v[3])};
    }
    *(i32x2_t*)p = w;
  }
}

// A wave's part of a result in rows: tile row r of the result is row r0 + r, present below `rows`; the
// columns start at c0, present below `cols` (a multiple of 8). Scaled by f, in o's type, added to or not. Returns whether all of it is
// present (then it took a store per piece of 16-bit results at least).
template <class S>
__device__ __forceinline__ bool store_tile(const OutArgs& o, f32x16_t (&acc)[S::MF][S::NF], float f, int64_t r0, int64_t rows, int c0, int cols,
                                           int lane, char* lds) {
#pragma unroll
  for (int j = 0; j < S::NF; ++j) {
    const int64_t rj = r0 + 32 * j;
    if (o.type == T_F32_ || o.accumulate) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        i32x4_t v[2 * S::MF];
        pieces32<S::MF>(j, h, v, [&](int i, int jj, int r) { return (int)f2u(acc[i][jj][r] * f); });
        put_rows<S::PIECES>(lds, lane, v, [&](int row, int c, i32x4_t x) {
          const int col = c0 + 16 * S::MF * h + 4 * c;
          if (rj + row < rows && col < cols) store4(o, rj + row, col, __builtin_bit_cast(f32x4_t, x));
        });
      }
    } else {
      i32x4_t v[2 * S::MF];
      if (o.type == T_BF16_) pieces16<S::MF>(acc, j, v, [f](float lo, float hi) { return pack16<MulBF16>(lo * f, hi * f); });
      else pieces16<S::MF>(acc, j, v, [f](float lo, float hi) { return pack16<MulF16>(lo * f, hi * f); });
      put_rows<S::PIECES>(lds, lane, v, [&](int row, int c, i32x4_t x) {
        const int col = c0 + 8 * c;
        if (rj + row < rows && col < cols) *(i32x4_t*)((uint16_t*)o.out + (rj + row) * o.ld + col) = x;
      });
    }
  }
  return r0 + S::WN_ROWS <= rows && c0 + S::WM_ROWS <= cols;
}

template <class S>
struct WeightJob : ProductArgs {
  static constexpr int STORES = S::NF * S::PIECES / 2;
  __device__ __forceinline__ void place(int u, int& dt, int& vt, int& slot) const {
    dt = u % d_tiles;
    slot = u / d_tiles % w_slots;
    vt = u / d_tiles / w_slots;
  }
  __device__ __forceinline__ TileUnit unit(int u) const {
    int dt, vt, slot;
    place(u, dt, vt, slot);
    const int64_t t0 = slot * w_per, left = N - t0, rows = left < w_per ? left : w_per;
    const int d0 = dt * S::M, v = vt * S::N;
    const int dc = D - d0 < S::M ? D - d0 : S::M;
    // (X's rows with the first number of G, then again with the second)
    const int stages = (int)((rows + 31) / 32);
    const char *x = X + t0 * ldx + 2 * d0, *g = G + t0 * ldg + 2 * (int64_t)v;
    return {{x, ldx, rows, 2 * dc, stages, x}, {g, ldg, rows, 2 * S::N, stages, g + N * ldg}, w_planes * stages};
  }
  __device__ __forceinline__ bool finish(int u, f32x16_t (&acc)[S::MF][S::NF], int wm, int wn, int lane, char* lds) const {
    int dt, vt, slot;
    place(u, dt, vt, slot);
    const int64_t c = (int64_t)vt * S::N + S::WN_ROWS * wn;
    const int d = dt * S::M + S::WM_ROWS * wm;
    const bool split = w_slots > 1;                        // (one call: the code of one)
    const OutArgs o = split ? OutArgs{wpart + (int64_t)slot * cols * D, D, T_F32_, 0} : dW;
    return store_tile<S>(o, acc, split ? 1.0f : *inv, split ? c : v0 + c, split ? cols : v1, d, D, lane, lds);
  }
};

template <class S>
struct FeatureJob : ProductArgs {
  static constexpr int STORES = S::NF * S::PIECES / 2;
  __device__ __forceinline__ void place(int u, int& dt, int& nt, int& slot) const {
    dt = u % d_tiles;
    nt = u / d_tiles % row_tiles;
    slot = u / d_tiles / row_tiles;                        // (units of one run share its weights)
  }
  __device__ __forceinline__ TileUnit unit(int u) const {
    int dt, nt, slot;
    place(u, dt, nt, slot);
    const int64_t c0 = slot * x_per, n = (int64_t)nt * S::N;
    const int64_t left = cols - c0, len = left < x_per ? left : x_per;
    const int d0 = dt * S::M, dc = D - d0 < S::M ? D - d0 : S::M;
    return {{W + (v0 + c0) * ldw + 2 * d0, ldw, v1 - v0 - c0, 2 * dc}, {G + n * ldg + 2 * c0, ldg, x_planes * N - n, 0}, (int)(len / 32)};
  }
  __device__ __forceinline__ bool finish(int u, f32x16_t (&acc)[S::MF][S::NF], int wm, int wn, int lane, char* lds) const {
    int dt, nt, slot;
    place(u, dt, nt, slot);
    const int64_t rows = x_planes * N;
    const OutArgs o = xpart ? OutArgs{xpart + slot * rows * D, D, T_F32_, !first} : dX;
    return store_tile<S>(o, acc, xpart ? 1.0f : *inv, (int64_t)nt * S::N + S::WN_ROWS * wn, rows, dt * S::M + S::WM_ROWS * wm, D, lane, lds);
  }
};

// A block takes the units of dW in turn with the others (the first w_units % blocks, the heavy ones, take one more),
// then x_light or x_heavy units of dX, so that both kinds of block end together: the light blocks go ahead by as
// many rounds as they have more. In a round neighbouring blocks have neighbouring units, which read the same
// rows of G (several units of a block in a row let each of them read G from memory again: 1.15 times longer).
// Blocks of an XCD have neighbouring numbers here.
template <class Mul, class S>
__global__ __launch_bounds__(S::THREADS, S::WAVES) void k_lin_products(ProductArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[S::lds(true)];
  const int blocks = (int)gridDim.x, per = blocks / 8;
  const int b = blocks % 8 == 0 ? ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3) : (int)blockIdx.x;
  {
    WeightJob<S> job;
    (ProductArgs&)job = a;
    tile_stream<Mul, true, true, S>(job, b, blocks, a.w_units, lds);
  }
  FeatureJob<S> job;
  (ProductArgs&)job = a;
  const int heavy = a.w_units % blocks, light = blocks - heavy;
  int ahead = (a.x_light - a.x_heavy) * light;
  if (ahead > a.x_units) ahead = a.x_units;
  for (int round = b < heavy ? 1 : 0; round < 2; ++round) {
    const int first = round ? ahead + b : b - heavy, step = round ? blocks : light;
    tile_stream<Mul, true, false, S>(job, first, step, round ? a.x_units : ahead, lds);
  }
}

// Rows [r0, r0 + rows) of a result from the partial sums of `slots` runs, `stride` floats apart. Thread (x, y) of a block of
// 64 x G sums the runs y, y + G, .. of vector x; the G sums are added in the order of y. Two results share a
// launch: the first `blocks` blocks take the first.
struct SumArgs { const float* part; int64_t stride, r0, rows; int slots, D; OutArgs o; };
template <int G>
__global__ __launch_bounds__(64 * G) void k_lin_sum(SumArgs a, SumArgs b, int blocks, const float* inv) {
  __shared__ f32x4_t sums[G][64];
  const int x = (int)threadIdx.x & 63, y = (int)threadIdx.x >> 6;
  const float f = *inv;
  const bool second = (int)blockIdx.x >= blocks;
  const SumArgs& s = second ? b : a;
  const int d4 = s.D / 4;
  const int64_t n4 = s.rows * d4, block = second ? blockIdx.x - blocks : blockIdx.x, all = second ? gridDim.x - blocks : blocks;
  for (int64_t i0 = block * 64; i0 < n4; i0 += all * 64) {
    const int64_t i = i0 + x;
    f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (i < n4) {
#pragma unroll 8
      for (int k = y; k < s.slots; k += G) v += *(const f32x4_t*)(s.part + k * s.stride + i * 4);
    }
    sums[y][x] = v;
    __syncthreads();
    if (y == 0 && i < n4) {
#pragma unroll
      for (int g = 1; g < G; ++g) v += sums[g][x];
      store4(s.o, s.r0 + i / d4, i % d4 * 4, v * f);
    }
    __syncthreads();
  }
}

// ---- launchers -------------------------------------------------------------------------------------
static unsigned sum_grid(int64_t rows, int D) {
  const int64_t want = ceil_div(rows * (D / 4), 64), cap = 32 * (int64_t)device_cus();
  return (unsigned)(want < cap ? want : cap);
}
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// The shape that takes N x V logits soonest.
static int logits_shape(int64_t N, int64_t V, int D, int cus, double* us) {
  int best = 0;
  for (int k = 0; k < SHAPE_COUNT; ++k) {
    const int m = SHAPES[k].size;
    const int64_t units = ceil_div(N, m) * ceil_div(V, m);
    const double t = units_time(SHAPES[k], units, D / 32, stage_time(SHAPES[k], units, cus), cus) + (double)N * V / m * 32e-6 / 5.0;   // (and the join)
    if (k == 0 || t < *us) {
      best = k;
      *us = t;
    }
  }
  return best;
}
LinearLayout linear_layout(int64_t N, int64_t V, int D, int M) {
  LinearLayout s{};
  double us;
  s.shape = logits_shape(N, V, D, device_cus(), &us);
  s.parts = 2 * ceil_div(V, SHAPES[s.shape].size);
  s.part = 0;
  s.given = up256((size_t)s.parts * N * 8);
  s.total = s.given + up256((size_t)N * (M > 0 ? M : 1) * 4);
  return s;
}

static LogitTiles tiles_of(int shape, const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t N, int64_t v0, int64_t v1, int D) {
  LogitTiles t{};
  t.X = (const char*)X; t.W = (const char*)W; t.ldx = 2 * ldx; t.ldw = 2 * ldw;
  t.N = N; t.v0 = v0; t.v1 = v1; t.stages = D / 32;
  t.row_tiles = (int)ceil_div(N, SHAPES[shape].size); t.label_tiles = (int)ceil_div(v1 - v0, SHAPES[shape].size);
  return t;
}

int run_linear_logprobs(const void* X, const void* W, int type, int64_t N, int64_t V, int D, int64_t ldx, int64_t ldw,
                        const int32_t* ids, int M, float* logp, float* row_max, float* log_sum, const LinearLayout& s,
                        void* workspace, hipStream_t st) {
  char* ws = (char*)workspace;
  StatArgs a{};
  a.t = tiles_of(s.shape, X, ldx, W, ldw, N, 0, V, D);
  a.ids = ids; a.M = M; a.part = (float2*)(ws + s.part); a.given = (float*)(ws + s.given);
  const unsigned grid = blocks_for(s.shape, (int64_t)a.t.row_tiles * a.t.label_tiles, device_cus());
  with_shape(s.shape, [&](auto shape) {
    typedef decltype(shape) S;
    if (type == T_BF16_) hipLaunchKernelGGL((k_lin_stats<MulBF16, S>), dim3(grid), dim3(S::THREADS), 0, st, a);
    else hipLaunchKernelGGL((k_lin_stats<MulF16, S>), dim3(grid), dim3(S::THREADS), 0, st, a);
  });
  if (hipGetLastError() != hipSuccess) return ELMO_EHIP_;
  int wide = 1;                                            // (few rows: more blocks, and more runs of parts in each)
  while (wide * 64 < N && wide < 16) wide *= 2;
  const int64_t most = MAX_THREADS / 1024;                 // blocks
  for (int64_t n0 = 0; n0 < N; n0 += most * wide) {
    const int64_t blocks = ceil_div(N - n0, wide);
    hipLaunchKernelGGL(k_lin_join, dim3((unsigned)(blocks < most ? blocks : most)), dim3(1024), 0, st, a.part, s.parts, n0, N, V, wide, ids,
                       M, a.given, logp, row_max, log_sum);
  }
  return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
}

// How one piece's products are spread over the device: the time (us) of a launch with dX in x_units units of x_stages
// stages and dW in w_units of w_stages, and how many units of dX a block takes that has one unit of dW more than the
// others (heavy) or not (light). add: dX's sums are added to those of the pieces before (20 us for 256 x 256). Within 5%
// of the times of 4096 x 131,072 x 768 in pieces of 16,384 to 131,072 labels and 4 to 8 runs.
static double products_time(const ShapeCost& c, int64_t w_units, int64_t w_stages, int64_t x_units, int64_t x_stages, bool add,
                            int cus, int* heavy, int* light) {
  const int64_t blocks = (int64_t)cus * c.blocks;
  const double stage = 1.1 * stage_time(c, w_units + x_units, cus);   // (K-major)
  const double tw = c.ends + (double)w_stages * stage, tx = c.ends + (add ? 20.0 * c.size * c.size / 65536.0 : 0.0) + (double)x_stages * stage;
  const int64_t rem = w_units % blocks;
  const double low = (double)(w_units / blocks) * tw, top = rem > 0 ? low + tw : low;
  *heavy = *light = 0;
  if (x_units == 0) return top;
  // the blocks end after m units of dX, counted from the end of dW's units of either kind: no earlier than the
  // work shared out evenly, and soon after that
  const double even = ((double)w_units * tw + (double)x_units * tx) / (double)blocks, from = even > top ? even : top;
  double best = 0.0;
  for (int k = 0; k < (rem > 0 ? 2 : 1); ++k) {
    const double start = k ? top : low;
    for (double m = (double)(int64_t)((from - start) / tx);; m += 1.0) {
      const double T = start + m * tx;
      if (best > 0.0 && T >= best) break;
      if (T < top) continue;
      const double h = rem > 0 ? (double)(int64_t)((T - top) / tx + 1e-6) : 0.0, l = (double)(int64_t)((T - low) / tx + 1e-6);
      if ((double)rem * h + (double)(blocks - rem) * l >= (double)x_units) {
        best = T;
        *heavy = (int)h;
        *light = (int)l;
        break;
      }
    }
  }
  return best;
}

// The piece (the caller's, or at most 2^27 gradient codes: 256 MiB, about the last-level cache), the shapes of its
// tiles and the runs, by the time they are expected to take: more pieces fill the device's last round better or
// worse, runs fill it with less in each, but are summed apart (dX by adding to memory, dW by another launch). Both
// products share a launch, or each has its own with its own shape (few rows, where memory bounds them: dW in the large
// shape, dX in the medium one take 156 us at 2 x 365,721 x 576, one launch 217; 93 and 139 at 64 x 131,072 x 768). dX goes
// first: the gradient codes' pass has just read W (behind dW: 210 and 133 us). One run over all labels in one plane
// needs no sum of dX and no launch for it (512 x 1,000 x 256, loss and gradient: 43 us against 46.5). The small shapes
// are tried at every size: with the large one alone from 1,024 rows and 16,384 labels on, gradients of few features take
// longer (4,096 x 32,003 x 64 191 us against 162, 2,698 x 120,686 x 128 551 against 507; of 114 sizes two were shorter so, by 5 and 8%
// at 320 features, and those of 768 and more did not change).
constexpr int64_t MAX_PIECE = (1 << 22) - 256;             // labels: 256 rows of G stay within 2^31 bytes
constexpr int64_t TWO_PLANES = 128;                        // rows up to which G is held as two numbers for every result
LinearGradLayout linear_grad_layout(int64_t N, int64_t V, int D, int M, int64_t chunk, ResultKind dx, ResultKind dw) {
  const bool need_dx = dx != NO_RESULT, need_dw = dw != NO_RESULT;
  LinearGradLayout s{};
  const int cus = device_cus();
  const int64_t whole = ceil_div(V, 256);   // pieces are multiples of 256 labels
  if (chunk > V) chunk = V;
  s.x_planes = N <= TWO_PLANES || dx == RESULT_32 ? 2 : 1;
  s.w_planes = N <= TWO_PLANES || dw == RESULT_32 ? 2 : 1;
  s.planes = (need_dx && s.x_planes == 2) || (need_dw && s.w_planes == 2) ? 2 : 1;
  int64_t most = chunk > 0 ? ceil_div(chunk, 256) : (int64_t(1) << 27) / (N <= TWO_PLANES ? N : s.planes * N) / 256;
  most = most < 1 ? 1 : (most > whole ? whole : most);
  if (most > MAX_PIECE / 256) most = MAX_PIECE / 256;
  const int64_t wst = ceil_div(N, 32), fewest = ceil_div(whole, most), x_rows = s.x_planes * N;
  const double rd = (double)x_rows * D * 4e-6 / 5.0;       // us for dX's partial sums to memory
  double least = 0.0;
  const int64_t last = chunk > 0 || fewest == 1 ? fewest : fewest + 4;
  for (int64_t pieces = fewest; pieces <= last && pieces <= whole; ++pieces) {
    const int64_t labels = (chunk > 0 ? most : ceil_div(whole, pieces)) * 256, used = ceil_div(V, labels);
    const int64_t n = labels < V ? labels : V, xst = ceil_div(n, 32);
    double logits;
    const int ls = logits_shape(N, n, D, cus, &logits);
    // each product by itself in its best shape and runs, and both in one launch of one shape
    struct Best { double us = 0.0; int shape = 0, slots = 1; } bw, bx;
    auto take = [&](double us, int w_shape, int x_shape, int64_t ws, int64_t xs) {
      us = (us + logits + 8.0) * (double)used;
      if (least > 0.0 && us >= least) return;
      least = us;
      s.piece = labels; s.x_slots = (int)xs; s.w_slots = (int)ws; s.logits = ls; s.w_shape = w_shape; s.x_shape = x_shape;
    };
    for (int k = 0; k < SHAPE_COUNT; ++k) {
      const ShapeCost& c = SHAPES[k];
      const int64_t dt = ceil_div(D, c.size), wt = need_dw ? ceil_div(n, c.size) * dt : 0, xt = need_dx ? ceil_div(x_rows, c.size) * dt : 0;
      const int64_t most_units = 2 * (int64_t)cus * c.blocks;
      int h, l;
      for (int64_t ws = 1; ws <= 16; ws *= 2) {
        if (ws > 1 && (!need_dw || N <= TWO_PLANES || ws * 2 > wst || wt * ws > most_units)) break;
        const double sum_w = ws > 1 ? 2.0 + (double)(ws + 1) * n * D * 4e-6 / 5.0 : 0.0;
        const int64_t w_stages = s.w_planes * ceil_div(wst, ws);
        if (need_dw) {
          const double us = products_time(c, wt * ws, w_stages, 0, 0, false, cus, &h, &l) + sum_w;
          if (bw.us == 0.0 || us < bw.us) bw = Best{us, k, (int)ws};
        }
        for (const int64_t xs : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 24, 32, 48, 64, 96, 128, 192, 256, 384, 512}) {
          if (xs > 1 && (!need_dx || xs * 4 > xst || xt * xs > most_units)) break;
          const double sum_x = s.x_planes == 1 && used == 1 && xs == 1 ? 0.0 : 5.0 + (double)xs * (rd + 0.02) / (double)used;   // (the sum of the runs: a launch more)
          if (need_dx && ws == 1) {
            const double us = products_time(c, 0, 0, xt * xs, ceil_div(xst, xs), used > 1, cus, &h, &l) + sum_x;
            if (bx.us == 0.0 || us < bx.us) bx = Best{us, k, (int)xs};
          }
          take(products_time(c, wt * ws, w_stages, xt * xs, ceil_div(xst, xs), used > 1, cus, &h, &l) + sum_w + sum_x, k, k, ws, xs);
        }
      }
    }
    if (need_dw && need_dx && bw.shape != bx.shape) take(bw.us + bx.us + 4.0, bw.shape, bx.shape, bw.slots, bx.slots);
  }
  s.x_per = ceil_div(ceil_div(s.piece < V ? s.piece : V, 32), s.x_slots) * 32;
  s.x_slots = (int)ceil_div(s.piece < V ? s.piece : V, s.x_per);
  s.w_per = ceil_div(wst, s.w_slots) * 32;
  s.w_slots = (int)ceil_div(N, s.w_per);
  s.sum_x = s.x_planes > 1 || s.x_slots > 1 || s.piece < V;
  size_t at = 0;
  s.most = at; at += up256(256 * 8);
  s.inv = at; at += 256;
  s.coef = at; at += up256((size_t)N * 8);
  s.up = at; at += up256((size_t)N * (M > 0 ? M : 1) * 4);
  s.G = at; at += up256((size_t)s.planes * N * s.piece * 2);
  s.xpart = at; if (need_dx && s.sum_x) at += up256((size_t)s.x_slots * x_rows * D * 4);
  s.wpart = at; if (need_dw && s.w_slots > 1) at += up256((size_t)s.w_slots * s.piece * D * 4);
  s.total = at;
  return s;
}

template <class Mul>
static int grad_as(const LinearGradCall& c, const LinearGradLayout& s, char* ws, hipStream_t st) {
  CoefArgs k{};
  k.N = c.N; k.V = c.V; k.M = c.M; k.ids = c.ids; k.row_max = c.row_max; k.log_sum = c.log_sum; k.dlogp = c.dlogp; k.dlse = c.dlse;
  k.most = (float2*)(ws + s.most); k.coef = (float2*)(ws + s.coef); k.up = (float*)(ws + s.up); k.inv = (float*)(ws + s.inv);
  k.f16 = std::is_same_v<Mul, MulF16>;
  // rows that every block can go through by itself need no launch for their bound
  k.parts = c.N * (c.M + 1) <= 16384 ? 0 : 256;
  if (k.parts) hipLaunchKernelGGL(k_lin_bound, dim3(k.parts), dim3(COEF_THREADS), 0, st, k);
  if (hipGetLastError() != hipSuccess) return ELMO_EHIP_;
  hipLaunchKernelGGL(k_lin_coef, dim3((unsigned)ceil_div(c.N, COEF_THREADS)), dim3(COEF_THREADS), 0, st, k);
  if (hipGetLastError() != hipSuccess) return ELMO_EHIP_;
  const int cus = device_cus();
  for (int64_t v0 = 0; v0 < c.V; v0 += s.piece) {
    const int64_t v1 = v0 + s.piece < c.V ? v0 + s.piece : c.V;
    GradArgs g{};
    g.t = tiles_of(s.logits, c.X, c.ldx, c.W, c.ldw, c.N, v0, v1, c.D);
    g.planes = s.planes; g.ids = c.ids; g.M = c.M; g.coef = k.coef; g.up = k.up; g.row_max = c.row_max; g.log_sum = c.log_sum; g.G = ws + s.G; g.ldg = 2 * s.piece;
    with_shape(s.logits, [&](auto shape) {
      typedef decltype(shape) S;
      const unsigned grid = blocks_for(s.logits, (int64_t)g.t.row_tiles * g.t.label_tiles, cus);
      hipLaunchKernelGGL((k_lin_grad_logits<Mul, S>), dim3(grid), dim3(S::THREADS), 0, st, g);
    });
    if (hipGetLastError() != hipSuccess) return ELMO_EHIP_;
    ProductArgs p{};
    p.X = (const char*)c.X; p.ldx = 2 * c.ldx; p.W = (const char*)c.W; p.ldw = 2 * c.ldw; p.G = ws + s.G; p.ldg = 2 * s.piece;
    p.w_planes = s.w_planes; p.x_planes = s.x_planes; p.N = c.N; p.v0 = v0; p.v1 = v1; p.D = c.D; p.inv = k.inv;
    p.cols = ceil_div(v1 - v0, 32) * 32;                   // (G is zero behind the last label, up to its tile's end)
    p.w_slots = s.w_slots; p.w_per = s.w_per; p.wpart = (float*)(ws + s.wpart);
    p.dW = OutArgs{c.dW, c.lddw, c.dw_type, c.accumulate};
    p.x_per = s.x_per; p.x_slots = (int)ceil_div(p.cols, s.x_per); p.first = v0 == 0;
    p.xpart = s.sum_x ? (float*)(ws + s.xpart) : nullptr; p.dX = OutArgs{c.dX, c.lddx, c.dx_type, 0};
    auto launch = [&](int number, bool dw, bool dx) {
      const ShapeCost& cost = SHAPES[number];
      ProductArgs q = p;
      q.d_tiles = (int)ceil_div(c.D, cost.size);
      q.row_tiles = (int)ceil_div(s.x_planes * c.N, cost.size);
      q.w_units = dw ? (int)ceil_div(v1 - v0, cost.size) * q.d_tiles * q.w_slots : 0;
      q.x_units = dx ? q.row_tiles * q.d_tiles * q.x_slots : 0;
      const unsigned grid = blocks_for(number, (int64_t)q.w_units + q.x_units, cus);
      if ((int64_t)q.w_units + q.x_units <= grid) q.x_light = 1;   // a unit for each block
      else products_time(cost, q.w_units, s.w_planes * ceil_div(s.w_per, 32), q.x_units, ceil_div(s.x_per, 32), s.piece < c.V, cus, &q.x_heavy, &q.x_light);
      with_shape(number, [&](auto shape) {
        typedef decltype(shape) S;
        hipLaunchKernelGGL((k_lin_products<Mul, S>), dim3(grid), dim3(S::THREADS), 0, st, q);
      });
      return hipGetLastError() == hipSuccess;
    };
    if (c.dW && c.dX && s.w_shape != s.x_shape) {
      if (!launch(s.x_shape, false, true) || !launch(s.w_shape, true, false)) return ELMO_EHIP_;
    } else if (!launch(c.dW ? s.w_shape : s.x_shape, c.dW != nullptr, c.dX != nullptr)) {
      return ELMO_EHIP_;
    }
    // the runs of dW summed, and those of dX behind the last piece
    SumArgs w{}, x{};
    if (c.dW && p.w_slots > 1) w = SumArgs{p.wpart, p.cols * c.D, v0, v1 - v0, p.w_slots, c.D, p.dW};
    if (c.dX && s.sum_x && v1 == c.V) x = SumArgs{p.xpart, c.N * c.D, 0, c.N, s.x_planes * s.x_slots, c.D, p.dX};
    const unsigned wb = w.rows ? sum_grid(w.rows, c.D) : 0, xb = x.rows ? sum_grid(x.rows, c.D) : 0;
    if (wb + xb == 0) continue;
    if (w.slots > 32 || x.slots > 32) hipLaunchKernelGGL(k_lin_sum<16>, dim3(wb + xb), dim3(1024), 0, st, w, x, (int)wb, (const float*)k.inv);
    else hipLaunchKernelGGL(k_lin_sum<4>, dim3(wb + xb), dim3(256), 0, st, w, x, (int)wb, (const float*)k.inv);
    if (hipGetLastError() != hipSuccess) return ELMO_EHIP_;
  }
  return ELMO_OK_;
}

// a gradient over no rows
__global__ __launch_bounds__(256) void k_lin_zero(OutArgs o, int64_t rows, int D) {
  const int d4 = D / 4;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < rows * d4; i += (int64_t)gridDim.x * 256)
    store4(o, i / d4, i % d4 * 4, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f});
}

int run_zero_rows(void* out, int type, int64_t rows, int D, int64_t ld, hipStream_t st) {
  const int64_t want = ceil_div(rows * (D / 4), 256), cap = 16 * (int64_t)device_cus();
  hipLaunchKernelGGL(k_lin_zero, dim3((unsigned)(want < cap ? want : cap)), dim3(256), 0, st, OutArgs{out, ld, type, 0}, rows, D);
  return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
}

int run_linear_logprobs_grad(const LinearGradCall& c, const LinearGradLayout& s, void* workspace, hipStream_t st) {
  return c.type == T_BF16_ ? grad_as<MulBF16>(c, s, (char*)workspace, st) : grad_as<MulF16>(c, s, (char*)workspace, st);
}

}  // namespace elmo
