// Device pieces shared by the operators: element types, activations and
// their slopes, wave sums.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "topk_device.hpp"
#include "topk_ops.hpp"

namespace tk {

struct bf16_t {
  uint16_t u;
};

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return __uint_as_float((uint32_t)v.u << 16); }
__device__ __forceinline__ float bits_f32(uint32_t h) { return __uint_as_float(h << 16); }

// Round to nearest even (the hardware conversion; NaN stays NaN).
__device__ __forceinline__ uint16_t bf16_bits(float v) {
  const __bf16 h = (__bf16)v;
  return __builtin_bit_cast(uint16_t, h);
}
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float v) { return bf16_t{bf16_bits(v)}; }

// 8 bf16 or 4 f32: one 16-byte vector of a row.
template <class T> struct Vec;
template <> struct Vec<float> {
  static constexpr int N = 4;
  __device__ static void load(const float* p, float* v) {
    const f32x4 q = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = q[i];
  }
  __device__ static void store(float* p, const float* v) {
    f32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = v[i];
    *reinterpret_cast<f32x4*>(p) = q;
  }
};
template <> struct Vec<bf16_t> {
  static constexpr int N = 8;
  __device__ static void load(const bf16_t* p, float* v) {
    const u32x4 q = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(q[i] << 16);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
    }
  }
  __device__ static void store(bf16_t* p, const float* v) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = (uint32_t)bf16_bits(v[2 * i]) | ((uint32_t)bf16_bits(v[2 * i + 1]) << 16);
    *reinterpret_cast<u32x4*>(p) = q;
  }
};

// VEC elements of a row that may end inside the vector: whole vectors when
// VEC is the 16-byte width, single elements when VEC is 1.
template <class T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float* v) {
  if constexpr (VEC == 1) v[0] = to_f32(p[0]);
  else Vec<T>::load(p, v);
}
template <class T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float* v) {
  if constexpr (VEC == 1) p[0] = from_f32<T>(v[0]);
  else Vec<T>::store(p, v);
}

// Activations in 32 bits.  Far left of zero gelu and silu are 0 and their
// slopes 0 (the formulas would give inf * 0 at -inf); NaN stays NaN.
template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (ACT == ACT_RELU) return z < 0.f ? 0.f : z;
  if constexpr (ACT == ACT_GELU) return z < -1e4f ? 0.f : 0.5f * z * erfcf(z * -0.70710678118654752f);
  if constexpr (ACT == ACT_SILU) return z < -1e4f ? 0.f : z / (1.f + expf(-z));
  return z;
}
template <int ACT>
__device__ __forceinline__ float slope_of(float z) {
  if constexpr (ACT == ACT_RELU) return z <= 0.f ? 0.f : 1.f;
  if constexpr (ACT == ACT_GELU) {
    const float s = 0.5f * erfcf(z * -0.70710678118654752f) +
                    z * expf(-0.5f * z * z) * 0.39894228040143268f;
    return z > 1e4f ? 1.f : (z < -1e4f ? 0.f : s);
  }
  if constexpr (ACT == ACT_SILU) {
    const float p = 1.f / (1.f + expf(-z));
    const float s = p * (1.f + z * (1.f - p));
    return z > 1e4f ? 1.f : (z < -1e4f ? 0.f : s);
  }
  return 1.f;
}

template <class V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

}  // namespace tk
