// Dropout whose mask is drawn from the counter-based generator of the stochastic rounding and never
// stored: y = r + s x for kept elements and r for dropped ones; the gradient draws the same mask again.
//
// Element i = first + t D + d of a call takes the 16 random bits of position i & 7 of block i >> 3, as the
// weights' update does (numerics.hpp), and is dropped if they are below limit = round(65536 p); the factor
// s = 65536 / (65536 - limit) is that of the probability in use, so that the expectation is exact.
//
// One Philox block (20 products, about 60 operations) serves 8 elements: 7 to 8 operations an element beside
// its 4 to 12 bytes, so that memory bounds it: 16,384 x 4,096 BF16 42.5 us (6.3 TB/s), with a residual 76 (5.3).
#include "lm_kernels.hpp"
#include "elem_types.hpp"

namespace elmo {

struct DropArgs {
  const void* x; const void* r; void* y;
  int64_t ldx, ldr, ldy, T, D;                             // T rows of D elements; pitches in elements
  uint64_t seed, step, first; const uint64_t* step_at;
  uint32_t limit; float factor;
};

template <typename E, bool RES>
__device__ __forceinline__ void drop8(const DropArgs& a, uint64_t step, const float* x, const float* r, uint64_t block, float* y) {
  const u32x4 draw = rng_block(a.seed, step, block);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = rng_pick(draw, i) >= a.limit ? x[i] * a.factor : 0.0f;
    y[i] = RES ? r[i] + v : v;
  }
}

// Rows whose 8-element vectors are blocks of the generator and 16-byte aligned (one long row where the
// tensors have no gaps). d8 = whole vectors of a row; what is left of the last row (below 8) is taken by the grid's
// first thread beside its own vectors.
template <typename E, bool RES>
__global__ __launch_bounds__(256) void k_dropout_rows(DropArgs a) {
  typedef typename E::raw raw;
  const uint64_t step = a.step + (a.step_at ? *a.step_at : 0);
  const int64_t d8 = a.D / 8, n8 = a.T * d8;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
    const int64_t t = a.T == 1 ? 0 : i / d8, d = (i - t * d8) * 8;
    float x[8], r[8], y[8];
    load_vec8<E>((const raw*)a.x + t * a.ldx + d, x);
    if constexpr (RES) load_vec8<E>((const raw*)a.r + t * a.ldr + d, r);
    drop8<E, RES>(a, step, x, r, (a.first + (uint64_t)(t * a.D + d)) >> 3, y);
    raw* p = (raw*)a.y + t * a.ldy + d;
#pragma unroll
    for (int h = 0; h < 8 / E::VEC; ++h) *(i32x4_t*)(p + h * E::VEC) = E::narrow(y + h * E::VEC);
  }
  if (a.D % 8 != 0 && blockIdx.x == 0 && threadIdx.x == 0) {   // (T = 1)
    const u32x4 draw = rng_block(a.seed, step, (a.first + (uint64_t)(d8 * 8)) >> 3);
    for (int64_t d = d8 * 8; d < a.D; ++d) {
      float v = rng_pick(draw, (int)(d & 7)) >= a.limit ? E::load((const raw*)a.x + d) * a.factor : 0.0f;
      if (RES) v = E::load((const raw*)a.r + d) + v;
      E::store((raw*)a.y + d, v);
    }
  }
}

// Any pitch and alignment: a thread takes the elements of one block of the generator, wherever they lie, one by one.
// 16,384 x 4,096, an element off their alignment: BF16 101 us (2.65 TB/s), FP32 342 (1.57), bound by those accesses; in
// whole vectors 38 and 96.
template <typename E, bool RES>
__global__ __launch_bounds__(256) void k_dropout_any(DropArgs a) {
  typedef typename E::raw raw;
  const uint64_t step = a.step + (a.step_at ? *a.step_at : 0);
  const uint64_t b0 = a.first >> 3, end = a.first + (uint64_t)(a.T * a.D), blocks = ((end + 7) >> 3) - b0;
  for (uint64_t i = blockIdx.x * (uint64_t)256 + threadIdx.x; i < blocks; i += (uint64_t)gridDim.x * 256) {
    const u32x4 draw = rng_block(a.seed, step, b0 + i);
    const uint64_t from = (b0 + i) * 8 < a.first ? a.first : (b0 + i) * 8;
    const uint64_t to = (b0 + i) * 8 + 8 < end ? (b0 + i) * 8 + 8 : end;
    int64_t t = (int64_t)((from - a.first) / (uint64_t)a.D), d = (int64_t)((from - a.first) - (uint64_t)(t * a.D));
    for (uint64_t e = from; e < to; ++e) {
      float v = rng_pick(draw, (int)(e & 7)) >= a.limit ? E::load((const raw*)a.x + t * a.ldx + d) * a.factor : 0.0f;
      if (RES) v = E::load((const raw*)a.r + t * a.ldr + d) + v;
      E::store((raw*)a.y + t * a.ldy + d, v);
      if (++d == a.D) { d = 0; ++t; }
    }
  }
}

template <typename E>
static void dropout_as(const DropArgs& a, bool rows, hipStream_t st) {
  const int64_t want = (a.T * a.D / 8 + 256) / 256, cap = 64 * (int64_t)device_cus();
  const dim3 grid((unsigned)(want < cap ? want : cap));
  if (rows) {
    if (a.r) hipLaunchKernelGGL((k_dropout_rows<E, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_dropout_rows<E, false>), grid, dim3(256), 0, st, a);
  } else {
    if (a.r) hipLaunchKernelGGL((k_dropout_any<E, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_dropout_any<E, false>), grid, dim3(256), 0, st, a);
  }
}

int run_dropout(const void* x, int type, int64_t T, int64_t D, int64_t ldx, const void* r, int64_t ldr, uint32_t limit,
                uint64_t seed, uint64_t step, const uint64_t* step_at, uint64_t first, void* y, int64_t ldy, hipStream_t st) {
  DropArgs a{};
  a.x = x; a.r = r; a.y = y; a.ldx = ldx; a.ldr = r ? ldr : ldx; a.ldy = ldy; a.T = T; a.D = D;
  a.seed = seed; a.step = step; a.step_at = step_at; a.first = first; a.limit = limit;
  a.factor = limit < 65536 ? 65536.0f / (65536.0f - (float)limit) : 0.0f;
  if (a.T == 1 || (a.ldx == D && a.ldr == D && a.ldy == D)) {  // no gaps: one long row
    a.D = a.T * a.D;
    a.T = 1;
    a.ldx = a.ldr = a.ldy = a.D;
  }
  const int64_t e = type == T_F32_ ? 4 : 2;
  auto vectors = [&](const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && (a.T == 1 || ld * e % 16 == 0); };
  const bool rows = first % 8 == 0 && (a.T == 1 || a.D % 8 == 0) && vectors(x, a.ldx) && vectors(y, a.ldy) && (!r || vectors(r, a.ldr));
  if (type == T_F32_) dropout_as<ElemF32>(a, rows, st);
  else if (type == T_BF16_) dropout_as<ElemBF16>(a, rows, st);
  else dropout_as<ElemF16>(a, rows, st);
  return hipGetLastError() == hipSuccess ? ELMO_OK_ : ELMO_EHIP_;
}

}  // namespace elmo
