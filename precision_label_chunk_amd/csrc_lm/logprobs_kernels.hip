// Log probabilities of given tokens under a row of logits, with the row's entropy and its top
// alternatives, and the gradient of the three with respect to the logits.
//
//   m = max_v z_v,  s = sum_v e^(z_v - m),  logp_j = (z_(id_j) - m) - log s,
//   H = -sum_v p_v log p_v = log s - (1/s) sum_v e^(z_v - m) (z_v - m).
//
// One pass over the logits: every lane carries the running maximum of its own elements and the two
// sums relative to it, rescaled when the maximum rises (in base 2: y = (z - m) log2 e), so that the
// row is read once and never stored. The maximum and log s stay apart (their sum is the row's log
// partition): at logits of large magnitude, such as a row masked with its type's lowest value, the
// rounded sum would lose log s.
//
// A block of 4 waves takes a contiguous segment of a row, each wave a contiguous quarter; short
// batches split every row over several blocks whose (m, s, t) and candidate keys a second kernel
// joins in a fixed order.
//
// Bound by HBM (medians of calls on logits that change from call to call): 4096 rows of 131072 BF16
// logits in 185 us (5.8 TB/s), 256 rows of 670000 FP32 logits in 118 us (5.8 TB/s). With alternatives the
// comparisons come close to the arithmetic that the read hides: top 5 of the FP32 rows 125 us, top 20 of
// the BF16 rows 194 us, top 64 225 us.
#include "elem_types.hpp"
#include "lm_kernels.hpp"
#include "wave_top.hpp"

namespace elmo {

constexpr int LP_WAVES = 4, LP_THREADS = 64 * LP_WAVES;
constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;

// a partial softmax: m the maximum, s = sum 2^y, t = sum 2^y y with y = (z - m) log2 e
struct SoftPart { float m, s, t; };

// the reference that exponents are taken against: the maximum, or 0 while nothing is above -inf
__device__ __forceinline__ float soft_ref(float m) { return m == -__builtin_inff() ? 0.0f : m; }

// moves a partial sum to the reference of the larger maximum mn
__device__ __forceinline__ void soft_move(SoftPart& a, float mn) {
  // d is -inf for an empty part or one that lies far below; 2^-1e4 is 0 as well, and d s stays finite
  // for every sum s of up to 2^31 elements, so that 0 times it is 0
  const float d = __builtin_fmaxf((a.m - soft_ref(mn)) * LOG2E, -1e4f);
  const float r = __builtin_amdgcn_exp2f(d);
  a.t = r * __builtin_fmaf(d, a.s, a.t);
  a.s *= r;
  a.m = mn;
}

// one element against the reference `ref`; a logit of -inf adds nothing to either sum
__device__ __forceinline__ void soft_add(SoftPart& a, float z, float ref) {
  const float y = (z - ref) * LOG2E;
  const float e = __builtin_amdgcn_exp2f(y);
  a.s += e;
  a.t = __builtin_fmaf(e, __builtin_fmaxf(y, -200.0f), a.t);   // 2^-200 is already 0 in binary32
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = __builtin_fmaxf(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ void wave_join(SoftPart& a) {
  soft_move(a, wave_max(a.m));
  a.s = wave_sum(a.s);
  a.t = wave_sum(a.t);
}

struct LogprobArgs {
  const void* Z; int64_t N, V, ldz;
  int64_t row0;                                 // the launch's first row
  const int32_t* ids; int M, k;
  float *logp, *entropy, *row_max, *log_sum;
  int32_t* top_idx; float* top_logp;
  int segs;                                     // blocks per row
  SoftPart* part; uint64_t* keys;               // [N][segs], [N][segs][k] (segs > 1)
};

// what the finished sums say of a row: log s and the entropy, both 0 where the mask leaves nothing
struct RowStats { float m, logs, H; bool empty; };
__device__ __forceinline__ RowStats row_stats(const SoftPart& a) {
  RowStats r;
  r.m = a.m;
  r.empty = a.m == -__builtin_inff() && a.s == 0.0f;
  r.logs = r.empty ? 0.0f : logf(a.s);
  r.H = r.empty ? 0.0f : __builtin_fmaf(-LN2, a.t / a.s, r.logs);
  return r;
}
__device__ __forceinline__ float row_logp(const RowStats& r, float z) {
  return r.empty ? -__builtin_inff() : (z - r.m) - r.logs;
}

// the outputs of row n, by one block, from its statistics and its k best keys in LDS
template <typename E>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t n, const SoftPart& sum, const uint64_t* keys) {
  const RowStats r = row_stats(sum);
  const int tid = (int)threadIdx.x;
  if (tid == 0) {
    a.entropy[n] = r.H;
    a.row_max[n] = r.m;
    a.log_sum[n] = r.logs;
  }
  const typename E::raw* z = (const typename E::raw*)a.Z + n * a.ldz;
  for (int j = tid; j < a.M; j += (int)blockDim.x) {
    const int32_t id = a.ids[n * a.M + j];
    float lp = 0.0f;                                        // a negative id stands for no token
    if (id >= 0) lp = id < a.V ? row_logp(r, E::load(z + id)) : __builtin_nanf("");
    a.logp[n * a.M + j] = lp;
  }
  if (tid < a.k) {
    const uint64_t q = keys[tid];                           // (best first)
    const uint32_t o = (uint32_t)(q >> 32);
    a.top_idx[n * a.k + tid] = (int32_t)~(uint32_t)q;
    a.top_logp[n * a.k + tid] = o == 0 ? __builtin_nanf("") : row_logp(r, value_of(o));
  }
}

// LDS of a block
template <bool TOP>
struct LogprobShared {
  uint64_t buf[TOP ? LP_WAVES : 1][TOP ? WaveTop::CAP : 1];
  uint64_t best[64];
  SoftPart sums[LP_WAVES];
  int cnts[LP_WAVES];
  uint32_t floors[LP_WAVES];                                // each wave's (k / 4)-th largest lane maximum
};

// joins the waves of a block: the sums into every thread, the k best keys, best first, into s.best
// (slots without a key: 0). `largest`: the order of the largest value among a lane's (0: none), for a
// last common bound, which few more than k keys reach; those rank by counting the larger ones.
template <bool TOP>
__device__ __forceinline__ void block_join(SoftPart& p, WaveTop& top, uint32_t largest, LogprobShared<TOP>& s) {
  const int wave = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  wave_join(p);
  if (lane == 0) s.sums[wave] = p;
  if constexpr (TOP) {
    if (top.cnt > WaveTop::MOST) top.cut();
    const uint32_t o[1] = {largest}, f = kth_of_lanes(o, (top.k + LP_WAVES - 1) / LP_WAVES);
    if (lane == 0) s.floors[wave] = f;
  }
  __syncthreads();
  SoftPart q = s.sums[0];
#pragma unroll
  for (int w = 1; w < LP_WAVES; ++w) q.m = __builtin_fmaxf(q.m, s.sums[w].m);
  const float m = q.m;
  q.m = s.sums[0].m;
  soft_move(q, m);
#pragma unroll
  for (int w = 1; w < LP_WAVES; ++w) {
    SoftPart o = s.sums[w];
    soft_move(o, m);
    q.s += o.s;
    q.t += o.t;
  }
  p = q;
  if constexpr (TOP) {
    uint32_t least = ~0u;
#pragma unroll
    for (int w = 0; w < LP_WAVES; ++w) least = s.floors[w] < least ? s.floors[w] : least;
    top.keep_from(least);
    if (lane == 0) s.cnts[wave] = top.cnt;
    __syncthreads();
    const uint64_t a = lane < top.cnt ? s.buf[wave][lane] : 0, b = 64 + lane < top.cnt ? s.buf[wave][64 + lane] : 0;
    int ra = 0, rb = 0, total = 0;
    for (int w = 0; w < LP_WAVES; ++w) {
      const int c = s.cnts[w];
      total += c;
#pragma unroll 4
      for (int i = 0; i < c; ++i) ra += s.buf[w][i] > a;
      if (top.cnt > 64)                                     // (of this wave: uniform)
        for (int i = 0; i < c; ++i) rb += s.buf[w][i] > b;
    }
    if (a && ra < top.k) s.best[ra] = a;
    if (b && rb < top.k) s.best[rb] = b;
    if ((int)threadIdx.x >= total && (int)threadIdx.x < top.k) s.best[threadIdx.x] = 0;
    __syncthreads();
  }
}

template <typename E, bool TOP>
__global__ __launch_bounds__(LP_THREADS) void k_logprobs(LogprobArgs a) {
  constexpr int VEC = E::VEC, U = 4;                        // U vectors of 16 bytes per lane in flight
  __shared__ LogprobShared<TOP> s;
  const int wave = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  const int64_t n = a.row0 + blockIdx.x / a.segs;
  const int seg = (int)(blockIdx.x % a.segs);
  const typename E::raw* z = (const typename E::raw*)a.Z + n * a.ldz;
  // the row as up to VEC - 1 single elements, nv aligned vectors, up to VEC - 1 single elements
  const int mis = (int)(((uintptr_t)z & 15u) / sizeof(typename E::raw));
  int head = mis ? VEC - mis : 0;
  if (head > a.V) head = (int)a.V;
  const int nv = (int)((a.V - head) / VEC);
  const int tail = (int)(a.V - head - (int64_t)nv * VEC);
  const i32x4_t* zv = (const i32x4_t*)(z + head);
  // this wave's vectors [v0, v1): whole steps of 64 vectors
  const int parts = a.segs * LP_WAVES, me = seg * LP_WAVES + wave;
  const int steps = (nv + 63) / 64, per = steps / parts, more = steps % parts;
  const int s0 = me * per + (me < more ? me : more), s1 = s0 + per + (me < more ? 1 : 0);
  const int v0 = s0 * 64, v1 = s1 * 64 < nv ? s1 * 64 : nv;

  const float ninf = -__builtin_inff();
  SoftPart p{ninf, 0.0f, 0.0f};
  WaveTop top;
  top.init(s.buf[TOP ? wave : 0], TOP ? a.k : 0);
  if constexpr (TOP) {
    if (threadIdx.x < LP_WAVES) s.floors[threadIdx.x] = 0;
    __syncthreads();
  }

  // single elements: lane l takes element e0 + l of c
  auto singles = [&](int64_t e0, int c) __attribute__((always_inline)) {
    const bool in = lane < c;
    const float v = in ? E::load(z + e0 + lane) : ninf;
    soft_move(p, __builtin_fmaxf(p.m, v));
    soft_add(p, v, soft_ref(p.m));
    if constexpr (TOP) {
      top.threshold(top.bound);
      top.push(in && top.wants(v), key_of(v, (uint32_t)(e0 + lane)));   // (at most 7: there is room)
    }
  };
  if (me == 0 && head) singles(0, head);

  uint32_t chunks = 1;
  auto chunk = [&](int v, auto whole) __attribute__((always_inline)) {
    i32x4_t r[U];
    float f[U][VEC], mx[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = v + 64 * u + lane;
      r[u] = i32x4_t{0, 0, 0, 0};
      if (whole || i < v1) r[u] = __builtin_nontemporal_load(zv + i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      E::widen(r[u], f[u]);
      if (!whole && v + 64 * u + lane >= v1) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[u][e] = ninf;
      }
      mx[u] = f[u][0];
#pragma unroll
      for (int e = 1; e < VEC; ++e) mx[u] = __builtin_fmaxf(mx[u], f[u][e]);
    }
    float mn = p.m;
#pragma unroll
    for (int u = 0; u < U; ++u) mn = __builtin_fmaxf(mn, mx[u]);
    soft_move(p, mn);
    const float ref = soft_ref(mn);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < VEC; ++e) soft_add(p, f[u][e], ref);
    if constexpr (TOP) {
      // (a maximum is one of the values; -inf says nothing: it may stand for none)
      auto order = [&](float x) __attribute__((always_inline)) { return x == ninf ? 0u : order_of(x); };
      uint32_t first = 0;
      if ((chunks & (chunks - 1)) == 0) {                   // after 1, 2, 4, .. chunks
        const uint32_t o[1] = {order(p.m)};
        if (chunks == 1) {                                  // (many alternatives: of the vectors' maxima)
          if (a.k <= 16) first = kth_of_lanes(o, a.k);
          else {
            uint32_t ou[U];
#pragma unroll
            for (int u = 0; u < U; ++u) ou[u] = order(mx[u]);
            first = kth_of_lanes(ou, a.k);
          }
        }
        if (v + 64 * U < v1) {                              // (the last chunk's would bound nothing)
          const uint32_t mine = kth_of_lanes(o, (a.k + LP_WAVES - 1) / LP_WAVES);
          if (lane == 0) __hip_atomic_store(&s.floors[wave], mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
      }
      ++chunks;
      uint32_t least = ~0u;
#pragma unroll
      for (int w = 0; w < LP_WAVES; ++w) {
        const uint32_t fw = __hip_atomic_load(&s.floors[w], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        least = fw < least ? fw : least;
      }
      // values of this chunk count if they reach the first bound or the waves' common one (which other
      // waves' values of larger indices may have set), and have to pass the wave's own
      const uint32_t reach = order_below(first > least ? first : least);
      top.threshold(reach > top.bound ? reach : top.bound);
      static_for<0, U>([&](auto u) __attribute__((always_inline)) {   // (register arrays: expanded at compile time)
        const int i = v + 64 * u + lane;
        const bool in = whole || i < v1;
        if (__ballot(in && top.wants(mx[u]))) top.push_all(in, f[u], (uint32_t)(head + VEC * i));
      });
      top.bound = first > top.bound ? first : top.bound;
    }
  };
  int v = v0;
  for (; v + 64 * U <= v1; v += 64 * U) chunk(v, std::true_type{});
  if (v < v1) chunk(v, std::false_type{});
  if (me == parts - 1 && tail) singles(a.V - tail, tail);

  block_join<TOP>(p, top, p.m == ninf ? 0u : order_of(p.m), s);
  if (a.segs == 1) {
    write_row<E>(a, n, p, s.best);
  } else {
    const int64_t at = n * a.segs + seg;
    if (threadIdx.x == 0) a.part[at] = p;
    if (TOP && (int)threadIdx.x < a.k) a.keys[at * a.k + threadIdx.x] = s.best[threadIdx.x];   // (0: no key)
  }
}

// joins the blocks of a row: part i by thread i % 256, then as the waves of a block
template <typename E, bool TOP>
__global__ __launch_bounds__(LP_THREADS) void k_logprobs_join(LogprobArgs a) {
  __shared__ LogprobShared<TOP> s;
  const int64_t n = blockIdx.x;
  SoftPart p{-__builtin_inff(), 0.0f, 0.0f};
  WaveTop top;
  top.init(s.buf[TOP ? threadIdx.x >> 6 : 0], TOP ? a.k : 0);
  for (int i = (int)threadIdx.x; i < a.segs; i += LP_THREADS) {
    SoftPart o = a.part[n * a.segs + i];
    const float m = __builtin_fmaxf(p.m, o.m);
    soft_move(p, m);
    soft_move(o, m);
    p.s += o.s;
    p.t += o.t;
  }
  uint32_t largest = 0;
  if constexpr (TOP) {
    const int total = a.segs * a.k;
    const uint64_t* keys = a.keys + n * total;
    const int lane = (int)(threadIdx.x & 63), i0 = (int)(threadIdx.x & ~63u);
    for (int i = (int)threadIdx.x; i < total; i += LP_THREADS) {
      const uint32_t o = (uint32_t)(keys[i] >> 32);
      largest = o > largest ? o : largest;
    }
    const uint32_t o[1] = {largest};
    if (total > 64 * LP_WAVES) top.threshold(order_below(kth_of_lanes(o, a.k)));
    for (int i = i0; i < total; i += LP_THREADS) {          // (in no order of their indices: a cut lets ties in)
      const uint64_t q = i + lane < total ? keys[i + lane] : 0;   // (0: a segment of fewer than k elements)
      top.push(q != 0 && top.wants(value_of((uint32_t)(q >> 32))), q);
      if (top.cnt > WaveTop::CAP - 64) top.cut();
    }
  }
  block_join<TOP>(p, top, largest, s);
  write_row<E>(a, n, p, s.best);
}

// ---- gradient ------------------------------------------------------------------------------------
// With upstream gradients g_j of logp_j, gH of H and gL of log s + m (the log partition):
//   dz_v = p_v (gL - sum_j g_j - gH (log p_v + H)) + sum_{j: id_j = v} g_j,
// p_v = 2^((z_v - m) log2 e - log2 s). Elementwise, bound by HBM (the logits read, the gradient
// written: 4096 x 131072 BF16 in 352 us, 6.1 TB/s, median). The few elements that a given token names are
// computed before the block's pass over its segment and written after it, so that dZ may be the logits' own memory; a token given more than
// once is summed in the order of its places, by the thread of its first.
struct LogprobGradArgs {
  const void* Z; int64_t N, V, ldz;
  int64_t row0;                                 // the launch's first row
  const int32_t* ids; int M;
  const float *row_max, *log_sum, *entropy, *dlogp, *dentropy, *dlse;
  void* dZ; int64_t ldd;
  int segs;
};

template <typename E, bool HAS_H>
__global__ __launch_bounds__(256) void k_logprobs_grad(LogprobGradArgs a) {
  constexpr int VEC = E::VEC, U = 4;
  typedef typename E::raw raw;
  const int tid = (int)threadIdx.x;
  const int64_t n = a.row0 + blockIdx.x / a.segs;
  const int seg = (int)(blockIdx.x % a.segs);
  const raw* z = (const raw*)a.Z + n * a.ldz;
  raw* d = (raw*)a.dZ + n * a.ldd;
  const float m = a.row_max[n], logs = a.log_sum[n], H = a.entropy[n];
  const bool empty = m == -__builtin_inff() && logs == 0.0f;   // the mask leaves nothing: the gradient is 0
  float c = a.dlse ? a.dlse[n] : 0.0f;
  const float gH = HAS_H ? a.dentropy[n] : 0.0f;
  for (int j = 0; j < a.M; ++j) {
    const int32_t id = a.ids[n * a.M + j];
    if (id >= 0) c -= id < a.V ? a.dlogp[n * a.M + j] : __builtin_nanf("");
  }
  const float ref = soft_ref(m), l2 = logs * LOG2E;
  const float cH = empty ? 0.0f : HAS_H ? __builtin_fmaf(-gH, H, c) : c, gL = empty ? 0.0f : -gH * LN2;
  auto log2p = [&](float zv) { return __builtin_fmaf(zv - ref, LOG2E, -l2); };
  auto factor = [&](float y) { return HAS_H ? __builtin_fmaf(gL, __builtin_fmaxf(y, -200.0f), cH) : cH; };
  // The exponential gives 0 below 2^-126, where p's factor may still lift the gradient above it: small
  // probabilities stay 2^64 times larger until they have met it (y + 64 is exact).
  auto grad = [&](float zv) {
    const float y = log2p(zv);
    const bool low = y < -96.0f;
    return __builtin_amdgcn_exp2f(low ? y + 64.0f : y) * factor(y) * (low ? 0x1p-64f : 1.0f);
  };
  // those of a vector, by the short way where no p lies between 2^-191 and 2^-95 (the long one for all: 35
  // against 33 us at 333 x 32003 FP32)
  auto grads = [&](float (&f)[VEC]) __attribute__((always_inline)) {
    float y[VEC], near = 1e30f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      y[e] = log2p(f[e]);
      near = __builtin_fminf(near, __builtin_fabsf(y[e] + 143.0f));
    }
    if (__builtin_expect(near < 48.0f, 0)) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = grad(f[e]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = __builtin_amdgcn_exp2f(y[e]) * factor(y[e]);
    }
  };

  const int mis = (int)(((uintptr_t)z & 15u) / sizeof(raw));
  const bool vec = (((uintptr_t)z ^ (uintptr_t)d) & 15u) == 0;
  int head = mis ? VEC - mis : 0;
  if (head > a.V || !vec) head = (int)a.V;                     // rows of different alignment: element by element
  const int nv = (int)((a.V - head) / VEC);
  const int tail = (int)(a.V - head - (int64_t)nv * VEC);
  const int per = nv / a.segs, more = nv % a.segs;
  const int v0 = seg * per + (seg < more ? seg : more), v1 = v0 + per + (seg < more ? 1 : 0);
  // the elements this block writes: [e0, e1), the single ones at the row's ends by its end blocks
  int64_t e0 = head + (int64_t)v0 * VEC, e1 = head + (int64_t)v1 * VEC, h0 = 0, h1 = 0, t0 = 0, t1 = 0;
  if (vec) {
    if (seg == 0) { h1 = head; e0 = 0; }
    if (seg == a.segs - 1) { t0 = a.V - tail; t1 = a.V; e1 = a.V; }
  } else {
    const int64_t q = a.V / a.segs, r = a.V % a.segs;
    h0 = e0 = seg * q + (seg < r ? seg : r);
    h1 = e1 = e0 + q + (seg < r ? 1 : 0);
  }

  float mine = 0.0f;
  int64_t at = -1;
  if (tid < a.M) {
    const int32_t id = a.ids[n * a.M + tid];
    if (id >= e0 && id < e1) {
      at = id;
      for (int j = 0; j < a.M; ++j) {
        if (a.ids[n * a.M + j] != id) continue;
        if (j < tid) at = -1;
        mine += a.dlogp[n * a.M + j];
      }
      mine = empty ? 0.0f : mine + grad(E::load(z + id));
    }
  }
  __syncthreads();

  const i32x4_t* zv = (const i32x4_t*)(z + head);
  i32x4_t* dv = (i32x4_t*)(d + head);
  auto one = [&](i32x4_t r, int i) {
    float f[VEC];
    E::widen(r, f);
    grads(f);
    __builtin_nontemporal_store(E::narrow(f), dv + i);
  };
  int i = v0 + tid;
  for (; i + 256 * (U - 1) < v1; i += 256 * U) {
    i32x4_t r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = __builtin_nontemporal_load(zv + i + 256 * u);
#pragma unroll
    for (int u = 0; u < U; ++u) one(r[u], i + 256 * u);
  }
  for (; i < v1; i += 256) one(__builtin_nontemporal_load(zv + i), i);
  for (int64_t e = h0 + tid; e < h1; e += 256) E::store(d + e, grad(E::load(z + e)));
  for (int64_t e = t0 + tid; e < t1; e += 256) E::store(d + e, grad(E::load(z + e)));
  if (a.M) {
    __syncthreads();
    if (at >= 0) E::store(d + at, mine);
  }
}

// ---- launchers -------------------------------------------------------------------------------------
// Blocks per row: enough to fill the device several times over, but at least 4096 elements each, and
// at most 512 (one 8600000-token row with the top 5: 24 us with 512 blocks, 39 with 2048, whose join
// is one block's work; 26 with 256).
static int row_segments(int64_t N, int64_t V, int target) {
  int64_t s = (target + N - 1) / N;
  const int64_t most = V / 4096 > 0 ? V / 4096 : 1;
  if (s > most) s = most;
  if (s > 512) s = 512;
  return (int)(s < 1 ? 1 : s);
}

LogprobLayout logprobs_layout(int64_t N, int64_t V, int k) {
  LogprobLayout s{};
  // (4 blocks per CU: 64 rows of 262144 FP32 with the top 20 in 27.5 us, 32 with 8 blocks and 36 with 1)
  s.segs = row_segments(N, V, 4 * device_cus());
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t o = at; at += (bytes + 255) & ~(size_t)255; return o; };
  if (s.segs > 1) {
    s.part = take((size_t)N * s.segs * sizeof(SoftPart));
    s.keys = take((size_t)N * s.segs * k * 8);
  }
  s.total = at ? at : 256;
  return s;
}

// A launch holds fewer than 2^32 threads: rows go in runs of at most 2^23 (several runs only where a row
// is one block, as split rows are few).
template <typename F>
static int row_runs(int64_t N, int segs, F&& launch) {
  constexpr int64_t MOST = int64_t(1) << 23;
  for (int64_t row0 = 0; row0 < N; row0 += MOST) {
    launch(row0, dim3((unsigned)((N - row0 < MOST ? N - row0 : MOST) * segs)));
    if (hipGetLastError() != hipSuccess) return ELMO_EHIP_;
  }
  return ELMO_OK_;
}

template <typename E>
static int launch_logprobs(LogprobArgs a, hipStream_t st) {
  const dim3 block(LP_THREADS);
  const int rc = row_runs(a.N, a.segs, [&](int64_t row0, dim3 grid) {
    a.row0 = row0;
    if (a.k)
      hipLaunchKernelGGL((k_logprobs<E, true>), grid, block, 0, st, a);
    else
      hipLaunchKernelGGL((k_logprobs<E, false>), grid, block, 0, st, a);
  });
  if (rc != ELMO_OK_) return rc;
  if (a.segs > 1) {
    if (a.k)
      hipLaunchKernelGGL((k_logprobs_join<E, true>), dim3((unsigned)a.N), block, 0, st, a);
    else
      hipLaunchKernelGGL((k_logprobs_join<E, false>), dim3((unsigned)a.N), block, 0, st, a);
    if (hipGetLastError() != hipSuccess) return ELMO_EHIP_;
  }
  return ELMO_OK_;
}

int run_logprobs(const void* Z, int ztype, int64_t N, int64_t V, int64_t ldz, const int32_t* ids, int M, int k,
                 float* logp, float* entropy, float* row_max, float* log_sum, int32_t* top_idx, float* top_logp,
                 const LogprobLayout& s, void* workspace, hipStream_t st) {
  LogprobArgs a{};
  a.Z = Z; a.N = N; a.V = V; a.ldz = ldz; a.ids = ids; a.M = M; a.k = k;
  a.logp = logp; a.entropy = entropy; a.row_max = row_max; a.log_sum = log_sum;
  a.top_idx = top_idx; a.top_logp = top_logp;
  a.segs = s.segs;
  a.part = (SoftPart*)((uint8_t*)workspace + s.part);
  a.keys = (uint64_t*)((uint8_t*)workspace + s.keys);
  switch (ztype) {
    case T_F32_: return launch_logprobs<ElemF32>(a, st);
    case T_BF16_: return launch_logprobs<ElemBF16>(a, st);
    default: return launch_logprobs<ElemF16>(a, st);
  }
}

template <typename E>
static int launch_grad(LogprobGradArgs a, hipStream_t st) {
  const dim3 block(256);
  return row_runs(a.N, a.segs, [&](int64_t row0, dim3 grid) {
    a.row0 = row0;
    if (a.dentropy)
      hipLaunchKernelGGL((k_logprobs_grad<E, true>), grid, block, 0, st, a);
    else
      hipLaunchKernelGGL((k_logprobs_grad<E, false>), grid, block, 0, st, a);
  });
}

int run_logprobs_grad(const void* Z, int ztype, int64_t N, int64_t V, int64_t ldz, const int32_t* ids, int M,
                      const float* row_max, const float* log_sum, const float* entropy, const float* dlogp,
                      const float* dentropy, const float* dlse, void* dZ, int64_t ldd, hipStream_t st) {
  LogprobGradArgs a{};
  a.Z = Z; a.N = N; a.V = V; a.ldz = ldz; a.ids = ids; a.M = M;
  a.row_max = row_max; a.log_sum = log_sum; a.entropy = entropy;
  a.dlogp = dlogp; a.dentropy = dentropy; a.dlse = dlse; a.dZ = dZ; a.ldd = ldd;
  // (many short blocks stream best: 128 per CU 350 us, 16 per CU 401, at 4096 x 131072 BF16)
  a.segs = row_segments(N, V, 128 * device_cus());
  switch (ztype) {
    case T_F32_: return launch_grad<ElemF32>(a, st);
    case T_BF16_: return launch_grad<ElemBF16>(a, st);
    default: return launch_grad<ElemF16>(a, st);
  }
}

}  // namespace elmo
