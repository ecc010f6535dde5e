// The k best (value, index) pairs of a stream of values that one wave reads in ascending order of
// their indices: value descending, then index ascending, NaN last.
//
// Candidates are 64-bit keys in a wave-private LDS buffer: the value as an order-preserving whole
// number in the upper half (NaN lowest), the complement of the index in the lower, so that keys are
// distinct and their order is the wanted one. A value is appended only if it can still belong to
// the k best: the buffer's k-th key so far bounds it from below. When the buffer is nearly full it
// is cut to its k best, which raises the bound; on values in no particular order n elements are cut
// about log(n) / log(CAP / k) times, so that nearly every vector is passed over by one comparison.
#pragma once
#include "numerics.hpp"

namespace elmo {

__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = f2u(v + 0.0f);                        // -0 counts as +0
  return v != v ? 0u : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {    // (o > 0)
  return u2f((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ uint64_t key_of(float v, uint32_t idx) { return ((uint64_t)order_of(v) << 32) | (uint32_t)~idx; }

__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// LDS written by some lanes of a wave is read by others: keep the accesses in program order
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

struct WaveTop {
  static constexpr int CAP = 256;                          // keys per wave (4 per lane at a cut)
  uint64_t* buf;                                           // LDS, CAP keys
  int k, cnt;
  bool open;                                               // no bound yet: everything is a candidate
  bool tie;                                                // a cut since begin_step: equal values may precede
  float bound;

  __device__ __forceinline__ void init(uint64_t* lds, int k_) {
    buf = lds; k = k_; cnt = 0; open = true; tie = false; bound = 0.0f;
  }
  // Values of one step arrive in no order of their indices, so equality with a bound set inside
  // the step does not exclude; values of later steps have larger indices than all kept ones.
  __device__ __forceinline__ void begin_step() { tie = false; }
  __device__ __forceinline__ bool wants(float v) const { return open || v > bound || (tie && v == bound); }

  // the wanted ones of the W values f of each lane (indices i0, i0 + 1, ..), one per lane and turn
  template <int W>
  __device__ __forceinline__ void push_all(bool in, const float (&f)[W], uint32_t i0) {
    uint32_t left = 0;
#pragma unroll
    for (int e = 0; e < W; ++e) left |= in && wants(f[e]) ? 1u << e : 0u;
    while (__ballot(left != 0)) {
      const uint32_t e = left ? (uint32_t)__builtin_ctz(left) : 0u;
      float v = f[0];
#pragma unroll
      for (int j = 1; j < W; ++j) {
        const float fj = f[j];                             // (read in both arms: the array stays in registers)
        v = e == (uint32_t)j ? fj : v;
      }
      push(left && wants(v), key_of(v, i0 + e));           // (a cut may have raised the bound)
      left &= left - 1;
    }
  }
  // one candidate per lane (where `want`); all lanes of the wave call it
  __device__ __forceinline__ void push(bool want, uint64_t key) {
    const uint64_t mask = __ballot(want);
    if (mask == 0) return;
    if (want) buf[cnt + lanes_below(mask)] = key;
    cnt += __popcll(mask);
    if (cnt > CAP - 64) cut();
  }

  // keep the k best of the cnt <= CAP keys
  __device__ __forceinline__ void cut() {
    wave_lds_fence();
    if (cnt > k) {
      const int lane = (int)(threadIdx.x & 63);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t q = 64 * j + lane < cnt ? buf[64 * j + lane] : 0;   // (0 is no key: ~index >= 2^31)
        hi[j] = (uint32_t)(q >> 32); lo[j] = (uint32_t)q;
      }
      // the k-th largest upper half, from its top bit down: the largest P that k keys reach
      uint32_t P = 0;
#pragma unroll 1
      for (uint32_t b = 0x80000000u; b; b >>= 1) {
        int c = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) c += __popcll(__ballot(hi[j] >= (P | b)));
        if (c >= k) P |= b;
      }
      int over = 0, equal = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        over += __popcll(__ballot(hi[j] > P));
        equal += __popcll(__ballot(hi[j] == P && lo[j] != 0));
      }
      // of the keys with that upper half, the k - over with the largest lower half (smallest index)
      uint32_t Q = 1;
      if (over + equal > k) {
        Q = 0;
#pragma unroll 1
        for (uint32_t b = 0x80000000u; b; b >>= 1) {
          int c = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) c += __popcll(__ballot(hi[j] == P && lo[j] >= (Q | b)));
          if (c >= k - over) Q |= b;
        }
      }
      wave_lds_fence();
      int at = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool keep = hi[j] > P || (hi[j] == P && lo[j] >= Q);
        const uint64_t mask = __ballot(keep);
        if (keep) buf[at + lanes_below(mask)] = ((uint64_t)hi[j] << 32) | lo[j];
        at += __popcll(mask);
      }
      cnt = at;
      open = P == 0;
      bound = value_of(P);
      tie = true;
    }
    wave_lds_fence();
  }
};

}  // namespace elmo
