// Matrix products in 8-bit integers with a scale for each row of both operands, and the quantisation that
// makes such rows.
//
// y[n, v] = sx[n] sw[v] sum_k x[n, k] w[v, k]: the sum is exact (D <= 65536 products of at most 2^14 stay
// within 2^30), so its split along K and its order change nothing; what rounds is its conversion, the two
// scales and the result. 16,384 x 4,096 x 4,096: 252 us, 2,190 TOP/s (the library's product into 32-bit sums 250).
#include "tile_shapes.hpp"

namespace elmo {

// ---- quantisation ----------------------------------------------------------------------------------
// q = the whole number nearest to 127 x / top (halves to even), scale = top / 127. The quotient comes from
// one product with 127 / top; within 2^-13 of a half, where its roundings (at most 127 x 1.5 x 2^-23 < 2^-15)
// could decide, 254 |x| is compared with (2 k + 1) top, both exact in binary64.
__device__ __forceinline__ int quantise(float x, float inv, float top) {
  const float r = x * inv, k = __builtin_rintf(r);
  const float off = __builtin_fabsf(r - k);
  if (__builtin_expect(off > 0.4998f, 0)) {
    const float lo = __builtin_floorf(__builtin_fabsf(r));
    // |r| lies near lo + 1/2 (or, where floor took the wrong side, near lo - 1/2 or lo + 3/2: not within 2^-13)
    const double a = 254.0 * (double)__builtin_fabsf(x), b = (2.0 * (double)lo + 1.0) * (double)top;
    int q = (int)lo;
    if (a > b || (a == b && (q & 1))) ++q;
    return x < 0.0f ? -q : q;
  }
  return (int)k;
}

// A row per group of G threads (a wave, or the block); a thread's first VECS vectors of 8 elements stay in
// registers between the maximum and the codes, the rest is read again. 16,384 x 4,096 BF16: 43 us, 4.7 TB/s.
template <typename E, int G>
__global__ __launch_bounds__(256) void k_i8_quantize(const typename E::raw* x, int64_t N, int D, int64_t ldx, int8_t* codes, float* scales) {
  constexpr int VECS = 4;
  __shared__ float tops[4];
  const int lane = (int)threadIdx.x % G;
  const int64_t n = G == 64 ? blockIdx.x * (int64_t)4 + threadIdx.x / 64 : (int64_t)blockIdx.x;
  if (n >= N) return;                                      // (a whole wave, or the whole block)
  const typename E::raw* row = x + n * ldx;
  float f[VECS][8];
  float top = 0.0f;
  bool bad = false;
  auto see = [&](const float* v) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = __builtin_fabsf(v[i]);
      bad |= !(a < __builtin_inff());
      top = fmaxf(top, a);
    }
  };
#pragma unroll
  for (int v = 0; v < VECS; ++v) {
    const int d = (v * G + lane) * 8;
    if (d < D) {
      load_vec8<E>(row + d, f[v]);
      see(f[v]);
    }
  }
  for (int d = (VECS * G + lane) * 8; d < D; d += G * 8) {
    float g[8];
    load_vec8<E>(row + d, g);
    see(g);
  }
  if (bad) top = __builtin_inff();
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor(top, k));
  if constexpr (G == 256) {
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  }
  // a row with a NaN or an infinity: no codes, its scale NaN. 127 / top may leave binary32's normal range for
  // rows under 2^-100: those are scaled up first, by a power of two
  const bool none = !(top < __builtin_inff());
  const bool tiny = top < 7.8886090522101181e-31f;
  const float up = tiny ? 1.2676506002282294e30f : 1.0f;
  const float t = top * up, inv = none || top == 0.0f ? 0.0f : 127.0f / t;
  auto put = [&](int d, const float* v) __attribute__((always_inline)) {
    int w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = none ? 0 : quantise(v[i] * up, inv, t);
      w[i / 4] |= (q & 255) << 8 * (i % 4);
    }
    *(i32x2_t*)(codes + n * D + d) = i32x2_t{w[0], w[1]};
  };
#pragma unroll
  for (int v = 0; v < VECS; ++v) {
    const int d = (v * G + lane) * 8;
    if (d < D) put(d, f[v]);
  }
  for (int d = (VECS * G + lane) * 8; d < D; d += G * 8) {
    float g[8];
    load_vec8<E>(row + d, g);
    put(d, g);
  }
  if (lane == 0) scales[n] = none ? __builtin_nanf("") : top / 127.0f;
}

template <typename E>
static void quantize_as(const void* x, int64_t N, int D, int64_t ldx, int8_t* codes, float* scales, hipStream_t st) {
  // a wave holds 2048 features of a row in registers, a block 8192
  const int64_t rows = D <= 2048 ? 4 : 1, most = MAX_THREADS / 256 * rows;
  for (int64_t n0 = 0; n0 < N; n0 += most) {
    const int64_t n = N - n0 < most ? N - n0 : most;
    const typename E::raw* p = (const typename E::raw*)x + n0 * ldx;
    const dim3 grid((unsigned)ceil_div(n, rows));
    if (rows == 4) hipLaunchKernelGGL((k_i8_quantize<E, 64>), grid, dim3(256), 0, st, p, n, D, ldx, codes + n0 * D, scales + n0);
    else hipLaunchKernelGGL((k_i8_quantize<E, 256>), grid, dim3(256), 0, st, p, n, D, ldx, codes + n0 * D, scales + n0);
  }
}

int run_i8_quantize(const void* x, int type, int64_t N, int D, int64_t ldx, int8_t* codes, float* scales, hipStream_t st) {
  if (type == T_F32_) quantize_as<ElemF32>(x, N, D, ldx, codes, scales, st);
  else if (type == T_BF16_) quantize_as<ElemBF16>(x, N, D, ldx, codes, scales, st);
  else quantize_as<ElemF16>(x, N, D, ldx, codes, scales, st);
  return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
}

// ---- products --------------------------------------------------------------------------------------
struct I8Args {
  const char* X; const char* W;
  const float* sx; const float* sw;
  void* Y; int64_t ldy;                                    // elements
  int64_t N, L; int D;
  int row_tiles, label_tiles, slots, per;                  // runs of K: `per` stages each
  int* part;                                               // [slots][N][L4]: whole sums of the runs
  int64_t L4;
};

typedef i32x4_t __attribute__((aligned(4))) i32x4_a4_t;
typedef i32x4_t __attribute__((aligned(2))) i32x4_a2_t;
typedef i32x2_t __attribute__((aligned(2))) i32x2_a2_t;

// four results of a row, labels v .. v + 3
template <typename E>
__device__ __forceinline__ void store_results(typename E::raw* p, int64_t left, const float* y) {
  if (left >= 4) {
    if constexpr (E::VEC == 4) {
      *(i32x4_a4_t*)p = E::narrow(y);
    } else {
      const float z[8] = {y[0], y[1], y[2], y[3], 0, 0, 0, 0};
      const i32x4_t w = E::narrow(z);
      *(i32x2_a2_t*)p = i32x2_t{w[0], w[1]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < left) E::store(p + i, y[i]);
  }
}
// a piece of 16 bytes of results, `left` of them present
template <typename E>
__device__ __forceinline__ void store_piece(typename E::raw* p, int64_t left, i32x4_t x) {
  if (left >= E::VEC) {
    if constexpr (E::VEC == 4) *(i32x4_a4_t*)p = x;
    else *(i32x4_a2_t*)p = x;
  } else {
    float y[8];
    E::widen(x, y);
#pragma unroll
    for (int i = 0; i < E::VEC - 1; ++i)
      if (i < left) E::store(p + i, y[i]);
  }
}
// scales of labels v .. v + 3, zero past the last
__device__ __forceinline__ f32x4_t scales4(const float* sw, int64_t v, int64_t L) {
  f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (v + i < L) s[i] = sw[v + i];
  return s;
}

constexpr int I8_GROUP = 8;

template <typename E, bool PARTS, class S>
struct I8Job : I8Args {
  __device__ __forceinline__ void place(int u, int& lt, int& nt, int& slot) const {
    const int tiles = row_tiles * label_tiles;
    slot = u / tiles;
    u %= tiles;
    const int group = I8_GROUP * row_tiles, g = u / group, r = u % group;
    const int wide = label_tiles - g * I8_GROUP < I8_GROUP ? label_tiles - g * I8_GROUP : I8_GROUP;
    nt = r / wide;
    lt = g * I8_GROUP + r % wide;
  }
  __device__ __forceinline__ TileUnit unit(int u) const {
    int lt, nt, slot;
    place(u, lt, nt, slot);
    const int64_t l = (int64_t)lt * S::M, n = (int64_t)nt * S::N;
    const int s0 = slot * per, all = D / STAGE_K, len = all - s0 < per ? all - s0 : per;
    return {{W + l * D + s0 * STAGE_K, D, L - l, 0}, {X + n * D + s0 * STAGE_K, D, N - n, 0}, len};
  }
  static constexpr int STORES = S::NF * S::PIECES / (PARTS || E::VEC == 4 ? 1 : 2);
  __device__ __forceinline__ bool finish(int u, i32x16_t (&acc)[S::MF][S::NF], int wm, int wn, int lane, char* lds) const {
    int lt, nt, slot;
    place(u, lt, nt, slot);
    const int64_t v0 = (int64_t)lt * S::M + S::WM_ROWS * wm, n0 = (int64_t)nt * S::N + S::WN_ROWS * wn;
    const int64_t left = L - v0;                           // (scales past the last label read as zero)
    const auto scales = buffer_rsrc(PARTS ? nullptr : sw + v0, PARTS ? 0 : 4 * (int)(left < 0 ? 0 : left < S::WM_ROWS ? left : S::WM_ROWS));
#pragma unroll
    for (int j = 0; j < S::NF; ++j) {
      const int64_t r0 = n0 + 32 * j;
      if constexpr (!PARTS) {                              // the results take the sums' place
        const float s = r0 + (lane & 31) < N ? sx[r0 + (lane & 31)] : 0.0f;
#pragma unroll
        for (int i = 0; i < S::MF; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const i32x4_t t = buffer_load16(scales, 16 * (8 * i + 2 * q + (lane >> 5)));
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][j][4 * q + k] = (int)f2u((float)acc[i][j][4 * q + k] * s * u2f((uint32_t)t[k]));
          }
      }
      if constexpr (PARTS || E::VEC == 4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          i32x4_t v[2 * S::MF];
          pieces32<S::MF>(j, h, v, [&](int i, int jj, int r) { return (int)acc[i][jj][r]; });
          put_rows<S::PIECES>(lds, lane, v, [&](int row, int c, i32x4_t x) {
            const int64_t n = r0 + row, l = v0 + 16 * S::MF * h + 4 * c;
            if (n >= N || l >= L) return;
            if constexpr (PARTS) *(i32x4_t*)(part + ((int64_t)slot * N + n) * L4 + l) = x;
            else store_piece<E>((typename E::raw*)Y + n * ldy + l, L - l, x);
          });
        }
      } else {
        i32x4_t v[2 * S::MF];
        pieces16<S::MF>(acc, j, v, [](int lo, int hi) {
          const float z[8] = {u2f((uint32_t)lo), u2f((uint32_t)hi), 0, 0, 0, 0, 0, 0};
          return E::narrow(z)[0];
        });
        put_rows<S::PIECES>(lds, lane, v, [&](int row, int c, i32x4_t x) {
          const int64_t n = r0 + row, l = v0 + 8 * c;
          if (n < N && l < L) store_piece<E>((typename E::raw*)Y + n * ldy + l, L - l, x);
        });
      }
    }
    return n0 + S::WN_ROWS <= N && left >= S::WM_ROWS;
  }
};

template <typename E, bool PARTS, class S>
__global__ __launch_bounds__(S::THREADS, S::WAVES) void k_i8_tiles(I8Args a) {
  __shared__ __attribute__((aligned(1024))) char lds[S::lds(true)];
  I8Job<E, PARTS, S> job;
  (I8Args&)job = a;
  const UnitRange r = xcd_units(a.label_tiles * a.row_tiles * a.slots);
  tile_stream<MulI8, false, false, S>(job, r.first, r.step, r.end, lds);
}

// the runs' sums joined, scaled and rounded
template <typename E>
__global__ __launch_bounds__(256) void k_i8_join(I8Args a) {
  const int64_t l4 = a.L4 / 4, stride = a.N * a.L4;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < a.N * l4; i += (int64_t)gridDim.x * 256) {
    const int64_t n = i / l4, v = i % l4 * 4;
    i32x4_t s = *(const i32x4_t*)(a.part + n * a.L4 + v);
    for (int k = 1; k < a.slots; ++k) s += *(const i32x4_t*)(a.part + k * stride + n * a.L4 + v);
    const f32x4_t t = scales4(a.sw, v, a.L);
    const float f = a.sx[n];
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = (float)s[k] * f * t[k];
    store_results<E>((typename E::raw*)a.Y + n * a.ldy + v, a.L - v, y);
  }
}

// Up to 32 rows: weights straight from memory to the matrix cores, 64 bytes of K per product, LT tiles of 16 labels a
// wave against all rows.
__device__ __forceinline__ i32x4_t mul_i8_16(i32x4_t a, i32x4_t b, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ void lds_barrier() {            // (loads to registers stay on their way)
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Many labels: a block's 4 waves share the rows in LDS, PANEL features at a time, and its 128 labels leave through
// LDS, 256 or 512 bytes of a row at a time. 3M labels x 768: 1 row 386 us (6.0 TB/s), 16 rows with FP32 results 490
// (5.1; with the rows read from the caches and results in 64-byte pieces 615); 32 rows x 1M, 16-bit results 165 (277).
constexpr int ROWS_LT = 2;
template <typename E, int NT>
__global__ __launch_bounds__(256) void k_i8_rows(I8Args a) {
  constexpr int LT = ROWS_LT, LABELS = 64 * LT, PANEL = 1024, XP = PANEL + 16, ROWS = 16 * NT, AHEAD = 8 / LT;
  typedef typename E::raw raw;
  constexpr int PITCH = LABELS + 16 / (int)sizeof(raw);    // of the results (and XP of the rows): 16 bytes apart in banks
  constexpr int BYTES = ROWS * XP > ROWS * PITCH * (int)sizeof(raw) ? ROWS * XP : ROWS * PITCH * (int)sizeof(raw);
  __shared__ __attribute__((aligned(16))) char lds[BYTES];
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t l0 = (int64_t)blockIdx.x * LABELS;
  const char* w[LT];
  i32x4_t acc[LT][NT];
#pragma unroll
  for (int i = 0; i < LT; ++i) {                           // labels past the last are the last one again; not stored
    const int64_t row = l0 + (wave * LT + i) * 16 + (lane & 15);
    w[i] = a.W + (row < a.L ? row : a.L - 1) * a.D + 16 * (lane >> 4);
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  }
  const char* xs = lds + (lane & 15) * XP + 16 * (lane >> 4);
  for (int d0 = 0; d0 < a.D; d0 += PANEL) {
    const int width = a.D - d0 < PANEL ? a.D - d0 : PANEL, pieces = width / 16;
    if (d0 > 0) lds_barrier();
    for (int p = tid; p < ROWS * pieces; p += 256) {
      const int r = p / pieces, c = p % pieces * 16;       // (rows past the last: zeros)
      *(i32x4_t*)(lds + r * XP + c) = r < a.N ? *(const i32x4_t*)(a.X + (int64_t)r * a.D + d0 + c) : i32x4_t{0, 0, 0, 0};
    }
    auto load = [&](int s, auto count, i32x4_t (&f)[LT][AHEAD]) __attribute__((always_inline)) {
      constexpr int C = count;
#pragma unroll
      for (int k = 0; k < C; ++k)
#pragma unroll
        for (int i = 0; i < LT; ++i) f[i][k] = *(const i32x4_t*)(w[i] + d0 + (s + k) * 64);
    };
    auto mul = [&](int s, auto count, i32x4_t (&f)[LT][AHEAD]) __attribute__((always_inline)) {
      constexpr int C = count;
#pragma unroll
      for (int k = 0; k < C; ++k)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const i32x4_t x = *(const i32x4_t*)(xs + j * 16 * XP + (s + k) * 64);
#pragma unroll
          for (int i = 0; i < LT; ++i) acc[i][j] = mul_i8_16(f[i][k], x, acc[i][j]);
        }
    };
    const int steps = width / 64;
    int s = 0;
    i32x4_t f[LT][AHEAD];
    constexpr std::integral_constant<int, AHEAD> many{};
    constexpr std::integral_constant<int, 1> one{};
    if (steps >= AHEAD) load(0, many, f);
    lds_barrier();
    for (; s + 2 * AHEAD <= steps; s += AHEAD) {           // the next ones are on their way while these are used
      i32x4_t g[LT][AHEAD];
      load(s + AHEAD, many, g);
      mul(s, many, f);
#pragma unroll
      for (int i = 0; i < LT; ++i)
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) f[i][k] = g[i][k];
    }
    if (steps >= AHEAD) {
      mul(s, many, f);
      s += AHEAD;
    }
    for (; s < steps; ++s) {
      load(s, one, f);
      mul(s, one, f);
    }
  }
  lds_barrier();
#pragma unroll
  for (int i = 0; i < LT; ++i) {
    const int c = (wave * LT + i) * 16 + 4 * (lane >> 4);  // the lane's first of four labels in the block
    const f32x4_t t = scales4(a.sw, l0 + c, a.L);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = 16 * j + (lane & 15);
      const float f = r < a.N ? a.sx[r] : 0.0f;
      float y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = (float)acc[i][j][k] * f * t[k];
      store_results<E>((raw*)lds + r * PITCH + c, 4, y);
    }
  }
  lds_barrier();
  constexpr int PIECES = LABELS / E::VEC;                  // of 16 bytes in a row
#pragma unroll
  for (int p = tid; p < ROWS * PIECES; p += 256) {
    const int r = p / PIECES, c = p % PIECES * E::VEC;
    if (r < a.N && l0 + c < a.L)
      store_piece<E>((raw*)a.Y + r * a.ldy + l0 + c, a.L - l0 - c, *(const i32x4_t*)((raw*)lds + r * PITCH + c));
  }
}

// Few labels: a block's KS waves share the K of one tile.
template <typename E, int NT, int KS>
__global__ __launch_bounds__(64 * KS) void k_i8_rows_split(I8Args a) {
  __shared__ i32x4_t sums[KS][NT][64];
  const int lane = (int)threadIdx.x & 63, ks = (int)threadIdx.x >> 6;
  const int64_t v0 = (int64_t)blockIdx.x * 16;
  const int steps = a.D / 64, s0 = steps * ks / KS, s1 = steps * (ks + 1) / KS;
  // rows past the last are the last one again; their results are not stored
  const int64_t row = v0 + (lane & 15) < a.L ? v0 + (lane & 15) : a.L - 1;
  const char* w = a.W + row * a.D + 16 * (lane >> 4);
  const char* x[NT];
  i32x4_t acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t n = 16 * j + (lane & 15);
    x[j] = a.X + (n < a.N ? n : a.N - 1) * a.D + 16 * (lane >> 4);
    acc[j] = i32x4_t{0, 0, 0, 0};
  }
  auto steps_of = [&](int s, auto count) __attribute__((always_inline)) {
    constexpr int C = count;                               // products whose operands are on their way together
    i32x4_t fw[C], fx[NT][C];
#pragma unroll
    for (int k = 0; k < C; ++k) {
      fw[k] = *(const i32x4_t*)(w + (s + k) * 64);
#pragma unroll
      for (int j = 0; j < NT; ++j) fx[j][k] = *(const i32x4_t*)(x[j] + (s + k) * 64);
    }
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j] = mul_i8_16(fw[k], fx[j][k], acc[j]);
  };
  constexpr int AHEAD = 8 / NT;
  int s = s0;
  for (; s + AHEAD <= s1; s += AHEAD) steps_of(s, std::integral_constant<int, AHEAD>{});
  if (AHEAD > 4 && s + 4 <= s1) { steps_of(s, std::integral_constant<int, 4>{}); s += 4; }
  if (s + 2 <= s1) { steps_of(s, std::integral_constant<int, 2>{}); s += 2; }
  if (s < s1) steps_of(s, std::integral_constant<int, 1>{});
#pragma unroll
  for (int j = 0; j < NT; ++j) sums[ks][j][lane] = acc[j];
  __syncthreads();
  if (ks != 0) return;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll 5
    for (int k = 1; k < KS; ++k) acc[j] += sums[k][j][lane];
  const int64_t v = v0 + 4 * (lane >> 4);
  if (v >= a.L) return;
  const f32x4_t t = scales4(a.sw, v, a.L);
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t n = 16 * j + (lane & 15);
    if (n < a.N) {
      const float f = a.sx[n];
      float y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = (float)acc[j][k] * f * t[k];
      store_results<E>((typename E::raw*)a.Y + n * a.ldy + v, a.L - v, y);
    }
  }
}

constexpr int I8_ROWS = 32;                                // rows that the streaming kernel takes

// The time of a stage by the blocks that share a compute unit (small tiles: 0.14 us alone, 0.22 and 0.5 with two and
// four). By the device's share, as for 16-bit products, 133 x 8,935 x 4,352 takes 25.3 us and 512 x 4,096 x 4,096 24.2;
// by this 19.8 and 20.8 (but gradients of 333 x 32,003 x 1,024 in 16 bits 148 instead of 143).
static const ShapeCost I8_SHAPES[SHAPE_COUNT] = {{LargeTiles::M, LargeTiles::BLOCKS, 5.5, 0.5, 0.8},
                                                 {MediumTiles::M, MediumTiles::BLOCKS, 3.5, 0.2, 0.58},
                                                 {SmallTiles::M, SmallTiles::BLOCKS, 2.5, 0.15, 0.52}};
static double i8_stage_time(const ShapeCost& c, int64_t units, int cus) {
  const int64_t each = ceil_div(units, cus);
  const double part = c.full / c.blocks, shared = part * (double)(each < c.blocks ? each : c.blocks);
  if (each > 1) return c.alone > shared ? c.alone : shared;
  return part > c.alone ? c.alone + (part - c.alone) * (double)units / cus : c.alone;
}

// The tile shape and the runs of K by the time they are expected to take; a run keeps 4 stages.
I8Layout i8_layout(int64_t N, int64_t L, int D) {
  I8Layout s{};
  s.slots = 1;
  s.per = D / STAGE_K;
  s.L4 = ceil_div(L, 4) * 4;
  if (N > I8_ROWS) {
    const int64_t all = D / STAGE_K;
    const int cus = device_cus();
    double least = 0.0;
    for (int k = 0; k < SHAPE_COUNT; ++k) {
      const ShapeCost& c = I8_SHAPES[k];
      const int64_t tiles = ceil_div(L, c.size) * ceil_div(N, c.size);
      for (int64_t slots = 1; slots <= 64; slots *= 2) {
        if (slots > 1 && (slots * 4 > all || tiles * slots > 2 * (int64_t)cus * c.blocks)) break;
        double us = units_time(c, tiles * slots, ceil_div(all, slots), i8_stage_time(c, tiles * slots, cus), cus);
        if (slots > 1) us += 3.0 + (double)(2 * slots) * N * L * 4e-6 / 5.0;
        if (least == 0.0 || us < least) {
          least = us;
          s.shape = k;
          s.per = (int)ceil_div(all, slots);
        }
      }
    }
    s.slots = (int)ceil_div(all, s.per);
  }
  s.total = s.slots > 1 ? (size_t)s.slots * N * s.L4 * 4 : 0;
  return s;
}

template <typename E>
static int matmul_as(I8Args& a, int shape, hipStream_t st) {
  if (a.N <= I8_ROWS) {
    const int64_t tiles = ceil_div(a.L, 16), cus = device_cus();
    // Rows shared by a block: for labels that fill the device several times over, fewer of them where the rows fit
    // one panel (131,072 labels, 16 rows x 768: 24 us against 30 split; 1 row x 4096: 113 against 90)
    if (tiles >= 64 * cus || (tiles >= 16 * cus && a.D <= 1024)) {
      const int64_t most = MAX_THREADS / 256 * (64 * ROWS_LT);
      for (int64_t l0 = 0; l0 < a.L; l0 += most) {
        I8Args b = a;
        b.W += l0 * a.D; b.sw += l0; b.Y = (typename E::raw*)a.Y + l0; b.L = a.L - l0 < most ? a.L - l0 : most;
        const dim3 grid((unsigned)ceil_div(b.L, 64 * ROWS_LT));
        if (a.N <= 16) hipLaunchKernelGGL((k_i8_rows<E, 1>), grid, dim3(256), 0, st, b);
        else hipLaunchKernelGGL((k_i8_rows<E, 2>), grid, dim3(256), 0, st, b);
      }
    } else {
      const dim3 grid((unsigned)tiles);
#define ELMO_I8_SPLIT(NT, KS) hipLaunchKernelGGL((k_i8_rows_split<E, NT, KS>), grid, dim3(64 * KS), 0, st, a)
      const bool few = tiles < 2 * cus;                    // (then 16 waves a tile fill it sooner than 4)
      if (a.N <= 16) {
        if (few) ELMO_I8_SPLIT(1, 16); else ELMO_I8_SPLIT(1, 4);
      } else {
        if (few) ELMO_I8_SPLIT(2, 16); else ELMO_I8_SPLIT(2, 4);
      }
#undef ELMO_I8_SPLIT
    }
    return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
  }
  const dim3 grid(blocks_for(shape, (int64_t)a.row_tiles * a.label_tiles * a.slots, device_cus()));
  with_shape(shape, [&](auto tiles) {
    typedef decltype(tiles) S;
    if (a.slots == 1) hipLaunchKernelGGL((k_i8_tiles<E, false, S>), grid, dim3(S::THREADS), 0, st, a);
    else hipLaunchKernelGGL((k_i8_tiles<ElemF32, true, S>), grid, dim3(S::THREADS), 0, st, a);
  });
  if (hipGetLastError() != hipSuccess) return ELMO_EHIP_;
  if (a.slots == 1) return ELMO_OK_;
  const int64_t want = ceil_div(a.N * (a.L4 / 4), 256), cap = 16 * (int64_t)device_cus();
  hipLaunchKernelGGL(k_i8_join<E>, dim3((unsigned)(want < cap ? want : cap)), dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
}

int run_i8_matmul(const int8_t* X, const float* sx, const int8_t* W, const float* sw, int64_t N, int64_t L, int D, void* Y,
                  int ytype, int64_t ldy, const I8Layout& s, void* workspace, hipStream_t st) {
  I8Args a{};
  a.X = (const char*)X; a.W = (const char*)W; a.sx = sx; a.sw = sw; a.Y = Y; a.ldy = ldy; a.N = N; a.L = L; a.D = D;
  a.row_tiles = (int)ceil_div(N, SHAPES[s.shape].size); a.label_tiles = (int)ceil_div(L, SHAPES[s.shape].size); a.slots = s.slots; a.per = s.per;
  a.part = (int*)workspace; a.L4 = s.L4;
  if (ytype == T_F32_) return matmul_as<ElemF32>(a, s.shape, st);
  if (ytype == T_BF16_) return matmul_as<ElemBF16>(a, s.shape, st);
  return matmul_as<ElemF16>(a, s.shape, st);
}

}  // namespace elmo
