// The k best (value, index) pairs of a stream of values that one wave reads in ascending order of
// their indices: value descending, then index ascending, NaN last.
//
// Candidates are 64-bit keys in a wave-private LDS buffer: the value as an order-preserving whole
// number in the upper half (NaN 0), the complement of the index in the lower, so that keys are
// distinct and their order is the wanted one. A value is appended only if it can still belong to the
// k best, that is if it is over a threshold:
//   * the k-th best key of the buffer when it was last cut to its k best;
//   * the k-th largest of the lanes' own maxima (k lanes reach it, so k values do), for the first
//     values;
//   * the smallest over the block's waves of the (k / 4)-th largest of its lanes' maxima: together the
//     waves hold k values that reach it. It follows the whole block's values and is published again
//     whenever a wave has seen twice as many.
// With it a 131072-value row has about one candidate for every three vectors of 512 values, and the
// rest are passed over by one comparison each.
#pragma once
#include "../csrc/numerics.hpp"

namespace elmo {

__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = f2u(v + 0.0f);                        // -0 counts as +0
  return v != v ? 0u : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// the value of an order; NaN for orders below that of -inf
__device__ __forceinline__ float value_of(uint32_t o) { return u2f((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o); }
// the next smaller order a value can have (that of -0 is never used)
__device__ __forceinline__ uint32_t order_below(uint32_t o) { return o == 0u ? 0u : o == 0x80000000u ? 0x7ffffffeu : o - 1u; }
__device__ __forceinline__ uint64_t key_of(float v, uint32_t idx) { return ((uint64_t)order_of(v) << 32) | (uint32_t)~idx; }

__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// LDS written by some lanes of a wave is read by others: keep the accesses in program order
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A P that k of the lanes' orders (W per lane; 0: none) reach: the largest with zeros in its low half,
// or one that exactly k reach; 0 if fewer than k are not 0. (The upper half tells values apart to one
// part in 256: enough for a bound, at half the steps.)
template <int W>
__device__ __forceinline__ uint32_t kth_of_lanes(const uint32_t (&o)[W], int k) {
  uint32_t P = 0;
#pragma unroll 1
  for (uint32_t b = 0x80000000u; b >= 0x10000u; b >>= 1) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) n += __popcll(__ballot(o[w] >= (P | b)));
    if (n >= k) P |= b;
    if (n == k) break;
  }
  return P;
}

struct WaveTop {
  static constexpr int CAP = 384, PER = CAP / 64;          // keys per wave, and per lane at a cut
  static constexpr int GROUP = 4;                          // values per lane between checks of the room
  static constexpr int MOST = CAP - 64 * GROUP;            // keys that may stay: 2 per lane
  uint64_t* buf;                                           // LDS, CAP keys
  int k, cnt;
  uint32_t bound;                                          // values of later indices matter if above this order
  float over;                                              // the threshold in force: NaN lets everything pass

  __device__ __forceinline__ void init(uint64_t* lds, int k_) {
    buf = lds; k = k_; cnt = 0; bound = 0; over = __builtin_nanf("");
  }
  __device__ __forceinline__ void threshold(uint32_t o) { over = value_of(o); }
  // (a NaN value passes any threshold; vectors are only looked at if a number in them does)
  __device__ __forceinline__ bool wants(float v) const { return !(v <= over); }

  // one candidate per lane (where `want`); the caller sees to the room
  __device__ __forceinline__ void push(bool want, uint64_t key) {
    const uint64_t mask = __ballot(want);
    if (mask == 0) return;
    if (want) buf[cnt + lanes_below(mask)] = key;
    cnt += __popcll(mask);
  }
  // the wanted ones of the W values f of each lane (indices i0, i0 + 1, ..)
  template <int W>
  __device__ __forceinline__ void push_all(bool in, const float (&f)[W], uint32_t i0) {
#pragma unroll
    for (int e = 0; e < W; ++e) {
      push(in && wants(f[e]), key_of(f[e], i0 + e));
      if (e % GROUP == GROUP - 1 && cnt > MOST) cut();
    }
  }

  // keep the keys of at least this order; cnt <= MOST
  __device__ __forceinline__ void keep_from(uint32_t least) {
    wave_lds_fence();
    const int lane = (int)(threadIdx.x & 63);
    const uint64_t a = lane < cnt ? buf[lane] : 0, b = 64 + lane < cnt ? buf[64 + lane] : 0;
    const bool ka = a != 0 && (uint32_t)(a >> 32) >= least, kb = b != 0 && (uint32_t)(b >> 32) >= least;
    const uint64_t ma = __ballot(ka), mb = __ballot(kb);
    wave_lds_fence();
    if (ka) buf[lanes_below(ma)] = a;
    if (kb) buf[__popcll(ma) + lanes_below(mb)] = b;
    cnt = __popcll(ma) + __popcll(mb);
    wave_lds_fence();
  }

  // Keep the k best of the cnt <= CAP keys. The new bound holds for values behind the present vector;
  // its own values that equal it (their indices may be smaller) are still let in.
  __device__ __forceinline__ void cut() {
    wave_lds_fence();
    if (cnt > k) {
      const int lane = (int)(threadIdx.x & 63);
      uint32_t hi[PER], lo[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const uint64_t q = 64 * j + lane < cnt ? buf[64 * j + lane] : 0;   // (0 is no key: ~index >= 2^31)
        hi[j] = (uint32_t)(q >> 32); lo[j] = (uint32_t)q;
      }
      // the k-th largest upper half, from its top bit down: the largest P that k keys reach (or, as soon
      // as there is one, a P that exactly k reach)
      uint32_t P = 0;
      int c = 0;
#pragma unroll 1
      for (uint32_t b = 0x80000000u; b && c != k; b >>= 1) {
        int n = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) n += __popcll(__ballot(hi[j] >= (P | b)));
        if (n >= k) { P |= b; c = n; }
      }
      // of the keys with that upper half, those with the largest lower halves (smallest indices)
      uint32_t Q = 1;
      if (c != k) {
        int above = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) above += __popcll(__ballot(hi[j] > P));
        Q = 0;
        c = 0;
#pragma unroll 1
        for (uint32_t b = 0x80000000u; b && c != k - above; b >>= 1) {
          int n = 0;
#pragma unroll
          for (int j = 0; j < PER; ++j) n += __popcll(__ballot(hi[j] == P && lo[j] >= (Q | b)));
          if (n >= k - above) { Q |= b; c = n; }
        }
      }
      wave_lds_fence();
      int at = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const bool keep = lo[j] != 0 && (hi[j] > P || (hi[j] == P && lo[j] >= Q));
        const uint64_t mask = __ballot(keep);
        if (keep) buf[at + lanes_below(mask)] = ((uint64_t)hi[j] << 32) | lo[j];
        at += __popcll(mask);
      }
      cnt = at;
      bound = P > bound ? P : bound;
      const float now = value_of(order_below(P));
      if (!(now <= over)) over = now;                      // (an open threshold is NaN, and so is `now` below -inf)
    }
    wave_lds_fence();
  }
};

}  // namespace elmo
