// Element types of the tensors of the language-model operators (FP32, BF16, FP16) and their 16-byte
// vectors: VEC elements per vector, widened to and rounded from binary32.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../csrc/mfma.hpp"
#include "../csrc/numerics.hpp"

namespace elmo {

struct ElemF32 {
  typedef float raw;
  static constexpr int VEC = 4;
  static __device__ __forceinline__ float load(const raw* p) { return *p; }
  static __device__ __forceinline__ void store(raw* p, float v) { *p = v; }
  static __device__ __forceinline__ void widen(i32x4_t v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = u2f((uint32_t)v[i]);
  }
  static __device__ __forceinline__ i32x4_t narrow(const float* f) {
    return i32x4_t{(int)f2u(f[0]), (int)f2u(f[1]), (int)f2u(f[2]), (int)f2u(f[3])};
  }
};

struct ElemBF16 {
  typedef uint16_t raw;
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float load(const raw* p) { return bf16_to_f32(*p); }
  static __device__ __forceinline__ void store(raw* p, float v) { *p = (raw)f32_to_bf16_rne(v); }
  static __device__ __forceinline__ void widen(i32x4_t v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = u2f((uint32_t)v[i] << 16);
      f[2 * i + 1] = u2f((uint32_t)v[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ i32x4_t narrow(const float* f) {
    return i32x4_t{(int)pack_bf16x2(f[0], f[1]), (int)pack_bf16x2(f[2], f[3]), (int)pack_bf16x2(f[4], f[5]),
                   (int)pack_bf16x2(f[6], f[7])};
  }
};

struct ElemF16 {
  typedef uint16_t raw;
  typedef _Float16 f16x2_v __attribute__((ext_vector_type(2)));
  typedef float f32x2_v __attribute__((ext_vector_type(2)));
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float load(const raw* p) { return (float)__builtin_bit_cast(_Float16, *p); }
  static __device__ __forceinline__ void store(raw* p, float v) { *p = __builtin_bit_cast(uint16_t, (_Float16)v); }
  static __device__ __forceinline__ void widen(i32x4_t v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int w = v[i];                                   // (a vector element is no object to bit_cast)
      const f16x2_v h = __builtin_bit_cast(f16x2_v, w);
      f[2 * i] = (float)h[0];
      f[2 * i + 1] = (float)h[1];
    }
  }
  static __device__ __forceinline__ i32x4_t narrow(const float* f) {
    i32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __builtin_bit_cast(int, __builtin_convertvector((f32x2_v){f[2 * i], f[2 * i + 1]}, f16x2_v));
    return v;
  }
};

}  // namespace elmo
