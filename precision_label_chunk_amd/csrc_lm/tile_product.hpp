// Matrix products in tiles, C[m, n] = sum_k A[m, k] B[n, k], for kernels that do something of their
// own with the sums of a tile (softmax statistics, a gradient, scales) instead of storing them.
//
// A block of 2 x WN waves computes tiles of 64 MF x 32 NF WN, a wave 32 MF x 32 NF of it in sums of 32 x 32. The depth goes
// in stages of 64 bytes of K per row (32 elements of 16 bits, 64 of 8), copied from memory to LDS without
// passing registers, NBUF - 1 stages ahead, one barrier a stage. The stages of a block's tiles follow each other
// without a break: the first stages of the next tile are on their way while the sums of the last one are used.
//
// An operand is K-contiguous (rows of m or n, its elements of a row along K) or K-major (rows of k, 16-bit
// elements along m or n, read from LDS by the transposing reads). Both take 64 bytes of LDS per row of m or n
// and stage. The copies write 16 bytes a lane in lane order, so what a lane fetches is permuted instead:
//   K-contiguous  row r's four 16-byte pieces at p = c ^ f(r), f(r) = (r >> 1 & 3) ^ (r >> 3 & 1): the 8
//                 rows that a read serves at once touch all 32 banks once, any 16 rows all 64 once
//   K-major       row k's 16-byte piece c at c ^ 2 X(k & 3), X = 0, 2, 5, 7 (rows of 128 bytes: 0, 1, 2, 3): the same
//                 for the 4 rows x 32 (64) bytes of a transposing read
// (no bank conflicts counted in either).
//
// What bounds it: at 4,096 x 16,384 x 4,096 the matrix cores are busy 67 to 73% of the cycles and the card lowers its
// clock to 1.5 GHz for it: logits with their softmax 1,243 TFLOP/s (the library's product alone: 1,533), 8-bit integers
// at 16,384 x 4,096 x 4,096 2,190 TOP/s (2,180 to 2,230). LDS is in use a quarter of the time. Two blocks of 128 x 256
// per compute unit, four waves of 128 x 128, more stages ahead, wave priorities and fixed orders of reads and
// products were built and are as fast or slower (down to 0.6 of the rate).
#pragma once
#include "elem_types.hpp"

namespace elmo {

typedef __attribute__((address_space(3))) char lds_char_t;

// The matrix instruction of an element type: 32 x 32 sums over 32 bytes of K per row, 16 bytes a lane
// (row lane % 32, the K half lane / 32).
struct MulBF16 {
  typedef s16x8_t frag;
  typedef f32x16_t acc;
  typedef float sum;
  static constexpr int BYTES = 2;
  static __device__ __forceinline__ acc mul(frag a, frag b, acc c) { return mfma_bf16(a, b, c); }
};
struct MulF16 {
  typedef s16x8_t frag;
  typedef f32x16_t acc;
  typedef float sum;
  static constexpr int BYTES = 2;
  static __device__ __forceinline__ acc mul(frag a, frag b, acc c) {
    typedef __attribute__((ext_vector_type(8))) _Float16 f16x8_v;
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_v, a), __builtin_bit_cast(f16x8_v, b), c, 0, 0, 0);
  }
};
typedef __attribute__((ext_vector_type(16))) int i32x16_t;
struct MulI8 {
  typedef i32x4_t frag;
  typedef i32x16_t acc;
  typedef int sum;
  static constexpr int BYTES = 1;
  static __device__ __forceinline__ acc mul(frag a, frag b, acc c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
  }
};

// One operand of a tile: where its first stage starts, and how far it reaches. K-contiguous: `rows` valid
// rows (of m or n) at pitch `ld` bytes. K-major: `rows` valid rows of k, of which `cols` bytes belong to
// the tile and the matrix. What lies outside reads as zero, or as other elements of the matrix where it
// reaches only sums that nobody uses. A K-major operand may go on behind `turn` stages at `second`, with the same
// rows and columns.
struct Operand { const char* at; int64_t ld; int64_t rows; int cols; int turn = 0; const char* second = nullptr; };
struct TileUnit { Operand a, b; int stages; };

constexpr int STAGE_K = 64;                                // bytes of K per stage

// The tile shapes. Large: 128 x 64 a wave, the fewest LDS reads per product, one block per compute unit (NBUF = 3:
// 4 and 5 are no faster, and 96 KiB leave room for results on their way out). Medium and small: less is left
// empty by few rows, more blocks share a compute unit, and a stage alone takes less time.
template <int MF_, int NF_, int WN_, int NBUF_, int BLOCKS_>
struct TileShape {
  static constexpr int MF = MF_, NF = NF_, WN = WN_, NBUF = NBUF_;
  static constexpr int BLOCKS = BLOCKS_;                   // per compute unit
  static constexpr int M = 64 * MF, N = 32 * NF * WN, THREADS = 128 * WN, WM_ROWS = 32 * MF, WN_ROWS = 32 * NF;
  static constexpr int WAVES = BLOCKS * THREADS / 256;     // per SIMD
  static constexpr int PIECES = 4 * MF;                    // 16-byte pieces of a wave's row of 16-bit results
  static constexpr int PUT = 32 * PIECES * 16;             // LDS bytes of a wave for results on their way out
  static constexpr int BUF = (M + N) * STAGE_K;
  static constexpr int lds(bool put) { return NBUF * BUF + (put ? 2 * WN * PUT : 0); }
};
typedef TileShape<4, 2, 4, 3, 1> LargeTiles;               // 256 x 256
typedef TileShape<2, 2, 2, 3, 2> MediumTiles;              // 128 x 128
typedef TileShape<1, 1, 2, 4, 4> SmallTiles;               // 64 x 64

__device__ __forceinline__ int kc_swizzle(int row) { return ((row >> 1) & 3) ^ ((row >> 3) & 1); }
template <int ROWS>
__device__ __forceinline__ int km_swizzle(int k) { const int r = k & 3; return ROWS == 64 ? 2 * r : 2 * (2 * r | (r >> 1)); }

// every wave of the block has all but its last N vector memory operations and all its LDS reads behind it
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Sixteen bytes a lane from `buf` at byte offset `off` to LDS at `to` + 16 lane (zeros past the buffer's end).
// In assembly, for the compiler's own form makes every transposing LDS read behind it wait for all copies
// (gradients of 4,096 x 16,384 x 4,096: 1.56 ms with these waits, 1.39 without). No register receives
// anything; wait_copies() counts the copies. Five wait states: an SGPR of `buf` may come from a vector instruction.
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t buf, int off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(off), "s"(buf) : "memory", "m0");
}

// One operand's copies: ROWS of m or n per stage, THREADS threads.
template <bool KM, int ROWS, int THREADS, int BYTES>
struct StageCopy {
  static constexpr int COPIES = ROWS * 4 / THREADS;        // 16-byte pieces per thread and stage
  static constexpr int KROWS = STAGE_K / BYTES;            // rows of k per stage
  static constexpr int PER_ROW = ROWS * BYTES / 16;        // K-major: pieces per row of k
  int off;                                                 // byte offset of the thread's first piece
  int step;                                                // and of the next one from it
  const char* at;                                          // the stage to be copied next
  int64_t left, ld;                                        // K-major: its valid rows of k and those behind it
  int cols, bytes;
  int turn; const char* second; int64_t rows;              // K-major: stages up to the second part, its place
  __device__ __forceinline__ void start(const Operand& o, int tid) {
    at = o.at;
    ld = o.ld;
    if constexpr (KM) {
      const int k = tid / PER_ROW, c = (tid % PER_ROW) ^ km_swizzle<ROWS>(k);
      off = k * (int)ld + c * 16;
      step = THREADS / PER_ROW * (int)ld;
      left = rows = o.rows;
      cols = o.cols;
      turn = o.turn;
      second = o.second;
    } else {
      const int r = tid / 4, c = (tid % 4) ^ kc_swizzle(r);
      off = r * (int)ld + c * 16;
      step = THREADS / 4 * (int)ld;
      const int n = o.rows < ROWS ? (int)o.rows : ROWS;
      bytes = n > 0 ? (n - 1) * (int)ld + STAGE_K : 0;
    }
  }
  // the copies of the next stage into the LDS bytes from `to` on (a wave's part of each starts at wave * 1024)
  __device__ __forceinline__ void copy(uint32_t to, bool live) {
    if constexpr (KM) {
      const int n = left < KROWS ? (int)left : KROWS;
      bytes = n > 0 ? (n - 1) * (int)ld + cols : 0;
    }
    const auto buf = buffer_rsrc(at, live ? bytes : 0);
#pragma unroll
    for (int i = 0; i < COPIES; ++i) copy16(buf, off + i * step, to + i * THREADS * 16);
    if constexpr (KM) {
      at += KROWS * ld;
      left -= KROWS;
      if (--turn == 0) {
        at = second;
        left = rows;
      }
    } else {
      at += STAGE_K;
    }
  }
};

// A wave's fragments of a stage: F of 32 rows each from row `first` on.
template <bool KM, int ROWS, int F, class Mul>
struct StageRead {
  int at[KM ? F : 1];
  __device__ __forceinline__ void start(int first, int lane) {
    if constexpr (KM) {
      // lane's place in a transposing read: group g of 16 lanes takes columns 16 (g & 1) .. + 16 and k rows
      // 8 (g >> 1) .. + 4 (then + 4 .. + 8); lane j of it supplies row j / 4, columns 4 (j % 4) .. + 4
      const int g = lane >> 4, j = lane & 15, k = 8 * (g >> 1) + (j >> 2);
      const int col = first + 16 * (g & 1) + 4 * (j & 3);
#pragma unroll
      for (int f = 0; f < F; ++f) at[f] = k * (ROWS * 2) + (((col + 32 * f) >> 3) ^ km_swizzle<ROWS>(k)) * 16 + (col & 7) * 2;
    } else {
      const int r = first + (lane & 31);
      at[0] = r * STAGE_K + ((lane >> 5) ^ kc_swizzle(r)) * 16;
    }
  }
  // half h of the stage
  __device__ __forceinline__ void read(const char* from, int h, typename Mul::frag* out) const {
#pragma unroll
    for (int f = 0; f < F; ++f) {
      if constexpr (KM) {
        const char* p = from + at[f] + h * 16 * ROWS * 2;
        out[f] = join(lds_read_tr16((const uint16_t*)p), lds_read_tr16((const uint16_t*)(p + 4 * ROWS * 2)));
      } else {
        out[f] = *(const typename Mul::frag*)(from + (at[0] ^ (32 * h)) + f * 32 * STAGE_K);
      }
    }
  }
};

// A wave's results, on their way to memory in rows: 32 rows of P pieces of 16 bytes, of which a lane holds pieces
// 2 k + lane / 32 of row lane % 32. They go through LDS of the wave's own, so that P lanes write a row's 16 P
// bytes: put(row, piece, value). Straight from the sums a store reaches 32 rows with 16 or 32 bytes in each: 131,072 x
// 768 16-bit results of next to no products took 146 us that way, 37 in rows.
template <int P, class F>
__device__ __forceinline__ void put_rows(char* lds, int lane, const i32x4_t (&v)[P / 2], F&& put) {
  asm volatile("" : "+v"(lane));                           // (no address is held across the products)
  const int r = lane & 31;
#pragma unroll
  for (int k = 0; k < P / 2; ++k) *(i32x4_t*)(lds + r * (16 * P) + (((2 * k + (lane >> 5)) ^ (r & (P - 1))) * 16)) = v[k];
#pragma unroll
  for (int k = 0; k < P / 2; ++k) {
    const int row = (64 / P) * k + lane / P, c = lane % P;
    put(row, c, *(const i32x4_t*)(lds + row * (16 * P) + ((c ^ (row & (P - 1))) * 16)));
  }
  sched_fence();                                           // (the next rows' values are not formed ahead: registers)
}

// A wave's rows of m of one column as 16-bit pieces for put_rows: a lane has 4 of every 8, and swaps with the lane
// of the other half, so that each holds 8. pack(lo, hi) rounds two sums.
template <int MF, class Acc, class Pack>
__device__ __forceinline__ void pieces16(const Acc& acc, int j, i32x4_t (&v)[2 * MF], Pack&& pack) {
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      int lo[2], hi[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        lo[k] = pack(acc[i][j][4 * q + 2 * k], acc[i][j][4 * q + 2 * k + 1]);
        hi[k] = pack(acc[i][j][4 * q + 4 + 2 * k], acc[i][j][4 * q + 5 + 2 * k]);
        auto s = __builtin_amdgcn_permlane32_swap(lo[k], hi[k], false, false);
        lo[k] = (int)s[0];
        hi[k] = (int)s[1];
      }
      v[2 * i + q / 2] = i32x4_t{lo[0], lo[1], hi[0], hi[1]};
    }
}
// and half h of them (16 MF rows of m) as 32-bit pieces, 4 rows of m in each: word(i, j, r) gives a sum's bits
template <int MF, class Word>
__device__ __forceinline__ void pieces32(int j, int h, i32x4_t (&v)[2 * MF], Word&& word) {
#pragma unroll
  for (int k = 0; k < 2 * MF; ++k) {
    const int t = 2 * MF * h + k, i = t / 4, q = 4 * (t % 4);
    v[k] = i32x4_t{word(i, j, q), word(i, j, q + 1), word(i, j, q + 2), word(i, j, q + 3)};
  }
}

// The products of the units first, first + step, .. below `end`; job.unit(u) describes a unit,
// job.finish(u, acc, wm, wn, lane, lds) uses its sums (lds: S::PUT bytes of the wave's own behind the buffers, if the
// block has them): acc[i][j][r] of wave (wm, wn) is row m = S::WM_ROWS wm + 32 i + 8 (r / 4) + 4 (lane / 32) + r % 4 and
// column n = S::WN_ROWS wn + 32 j + lane % 32 of the tile. It returns whether the wave has issued at least Job::STORES
// stores (the same for all its lanes). Every unit has at least one stage. All threads of the block call it.
template <class Mul, bool AKM, bool BKM, class S, class Job>
__device__ __forceinline__ void tile_stream(const Job& job, int first, int step, int end, char* lds) {
  constexpr int THREADS = S::THREADS, NBUF = S::NBUF, WN = S::WN, A_BYTES = S::M * STAGE_K, BUF = S::BUF;
  typedef typename Mul::frag frag;
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  if (first >= end) return;

  StageCopy<AKM, S::M, THREADS, Mul::BYTES> ca;
  StageCopy<BKM, S::N, THREADS, Mul::BYTES> cb;
  constexpr int COPIES = decltype(ca)::COPIES + decltype(cb)::COPIES;
  int lu = first, ls = 0, lstages;                         // the unit and stage to be copied next
  int fill = 0;                                            // and its buffer
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char_t*)lds + wave * 1024;
  {
    const TileUnit t = job.unit(lu);
    ca.start(t.a, tid);
    cb.start(t.b, tid);
    lstages = t.stages;
  }
  auto fetch = [&]() __attribute__((always_inline)) {
    const uint32_t to = lds0 + fill * BUF;
    ca.copy(to, lu < end);                                 // (past the last unit: copies of nothing, for the count)
    cb.copy(to + A_BYTES, lu < end);
    fill = fill + 1 == NBUF ? 0 : fill + 1;
    if (++ls == lstages) {
      ls = 0;
      lu += step;
      if (lu < end) {
        const TileUnit t = job.unit(lu);
        ca.start(t.a, tid);
        cb.start(t.b, tid);
        lstages = t.stages;
      }
    }
  };

  StageRead<AKM, S::M, S::MF, Mul> ra;
  StageRead<BKM, S::N, S::NF, Mul> rb;
  ra.start(S::WM_ROWS * wm, lane);
  rb.start(S::WN_ROWS * wn, lane);
  frag fa[2][S::MF], fb[2][S::NF];
  typename Mul::acc acc[S::MF][S::NF];
  auto products = [&](int h) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < S::MF; ++i)
#pragma unroll
      for (int j = 0; j < S::NF; ++j) acc[i][j] = Mul::mul(fa[h][i], fb[h][j], acc[i][j]);
  };
  auto frags = [&](const char* from, int h) __attribute__((always_inline)) {
    rb.read(from + A_BYTES, h, fb[h]);
    ra.read(from, h, fa[h]);
  };

#pragma unroll
  for (int s = 0; s < NBUF - 1; ++s) fetch();
  int use = 0;
  // stage: its copies have landed (this wave's by the count, the others' by the barrier), and every wave has
  // read the buffer that the next copies go to; the last half's products run while its fragments are read
  // (behind a unit's end its stores are younger than the copies of the next NBUF - 1 stages: they need not be
  // waited for. job.finish says whether this wave has made all of its STORES.)
  auto stage = [&](bool go_on, bool stores) __attribute__((always_inline)) {
    if (stores) wait_copies<COPIES*(NBUF - 2) + Job::STORES>();
    else wait_copies<COPIES*(NBUF - 2)>();
    const char* from = lds + use * BUF;
    use = use + 1 == NBUF ? 0 : use + 1;
    frags(from, 0);
    if (go_on) products(1);
    frags(from, 1);
    fetch();                                               // (behind the reads: 3% faster than before them)
    products(0);
  };
  bool stored = false;
  for (int u = first; u < end; u += step) {
    const int stages = job.unit(u).stages;
#pragma unroll
    for (int i = 0; i < S::MF; ++i)
#pragma unroll
      for (int j = 0; j < S::NF; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
    stage(false, stored);
    int s = 1;
    for (; s < NBUF - 1 && s < stages; ++s) stage(true, stored);
    for (; s < stages; ++s) stage(true, false);
    products(1);
    stored = job.finish(u, acc, wm, wn, lane, lds + NBUF * BUF + wave * S::PUT);
  }
  wait_copies<0>();                                        // no copy is on its way when the block's LDS is given back
}

// Blocks go to the 8 XCDs in turn; each XCD gets a run of the units, which its blocks take in turn, so
// that units next to each other share an L2. (first, step, end) of this block's.
struct UnitRange { int first, step, end; };
__device__ __forceinline__ UnitRange xcd_units(int units) {
  const int n = (int)gridDim.x, b = (int)blockIdx.x;
  if (n < 8) return {b, n, units};
  const int xcd = b & 7, per = units / 8, more = units % 8;
  const int start = xcd * per + (xcd < more ? xcd : more), len = per + (xcd < more);
  return {start + (b >> 3), (n - xcd + 7) / 8, start + len};
}

}  // namespace elmo
