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

// 8 bf16 or 4 f32: one 16-byte vector of a row.  Vectors are read and written
// whole at any element alignment (global memory takes them; a row of odd length
// costs a little more than an aligned one, and no more instructions).
__device__ __forceinline__ u32x4 read16(const void* p) {
  u32x4 q;
  __builtin_memcpy(&q, p, 16);
  return q;
}

// The same, of what is read once: it does not push out what others read again.
__device__ __forceinline__ u32x4 read16_once(const void* p) {
  typedef u32x4 any_u32x4 __attribute__((aligned(2)));
  return __builtin_nontemporal_load(static_cast<const any_u32x4*>(p));
}

template <class T> struct Vec;
template <> struct Vec<float> {
  static constexpr int N = 4;
  __device__ static void unpack(u32x4 q, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(q[i]);
  }
  __device__ static u32x4 pack(const float* v) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __float_as_uint(v[i]);
    return q;
  }
  __device__ static void load(const float* p, float* v) { unpack(read16(p), v); }
  __device__ static void store(float* p, const float* v) {
    const u32x4 q = pack(v);
    __builtin_memcpy(p, &q, 16);
  }
};
template <> struct Vec<bf16_t> {
  static constexpr int N = 8;
  __device__ static void unpack(u32x4 q, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(q[i] << 16);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
    }
  }
  __device__ static u32x4 pack(const float* v) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = (uint32_t)bf16_bits(v[2 * i]) | ((uint32_t)bf16_bits(v[2 * i + 1]) << 16);
    return q;
  }
  __device__ static void load(const bf16_t* p, float* v) { unpack(read16(p), v); }
  __device__ static void store(bf16_t* p, const float* v) {
    const u32x4 q = pack(v);
    __builtin_memcpy(p, &q, 16);
  }
};

// The first of the VEC columns that a lane takes whose share begins at column
// c: a row's last vector begins earlier, so that it ends with the row, and its
// first columns are computed twice, the same both times.
template <int VEC>
__device__ __forceinline__ uint32_t column_of(uint32_t c, uint32_t d) {
  if constexpr (VEC == 1) return c;
  return c + VEC <= d ? c : d - VEC;   // d >= VEC
}

// VEC elements of a row: the 16-byte width, or 1.
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

// Rows that are moved, not computed: VEC elements of a row by their bits (a
// type's own load and store may quiet a NaN).
template <class U, int VEC> struct Bits {
  typedef u32x4 type;
  __device__ static type load(const U* p) { return read16(p); }
  __device__ static type load_once(const U* p) { return read16_once(p); }
  __device__ static type zero() { return u32x4{0, 0, 0, 0}; }
  __device__ static void store(U* p, type v) { __builtin_memcpy(p, &v, 16); }
  __device__ static void stream(U* p, type v) {
    typedef u32x4 any_u32x4 __attribute__((aligned(2)));
    __builtin_nontemporal_store(v, reinterpret_cast<any_u32x4*>(p));
  }
};
template <class U> struct Bits<U, 1> {
  typedef U type;
  __device__ static type load(const U* p) { return *p; }
  __device__ static type load_once(const U* p) { return *p; }
  __device__ static type zero() { return 0; }
  __device__ static void store(U* p, type v) { *p = v; }
  __device__ static void stream(U* p, type v) { *p = v; }
};

// Outputs from 16 MB on are stored past the caches: they would push out what
// the rest of the launch reads (the product of 4096 x 512 x 65536 bf16, in its
// first form 358 us against 439; the encoder's gradient at 65536 latents 92.6
// against 96.9).  Smaller ones stay for whoever reads them next.
constexpr int64_t STREAM_BYTES = int64_t(16) << 20;

// A whole vector past the caches.
template <class T>
__device__ __forceinline__ void stream_vec(T* p, const float* v) {
  typedef u32x4 any_u32x4 __attribute__((aligned(2)));
  __builtin_nontemporal_store(Vec<T>::pack(v), reinterpret_cast<any_u32x4*>(p));
}

// Activations in 32 bits.  Far left of zero gelu and silu are 0 and their
// slopes 0 (the formulas would give inf * 0 at -inf); NaN stays NaN.
//
// Results that are rounded to bf16 (T = bf16_t) use the hardware's exponential
// and reciprocal and, for the normal distribution function, a form of six
// terms; 32-bit results use the full functions.
//
// tail_of: 1 - Phi(|z|) and exp(-z^2 / 2).  With x = |z| / sqrt(2) the first is
// erfc(x) / 2 = exp(-x^2) P(t) / 2, t = 1 / (1 + 0.42 x), P without a constant
// term.  P's coefficients are the least-maximum fit (a linear program over 6000
// points of 0 <= x <= 40) of erfc(x) exp(x^2) to an error that is at most 2e-4
// of the value and 1e-7 of 1: left of zero gelu is z times this alone, so what
// counts there is the error relative to it.  Evaluated in 32 bits it is off by
// at most 1.8e-4 of its value, a tenth of the smallest half step of bf16, and
// by 2.7e-7 in all (form 7.1.26 of Abramowitz and Stegun, one term shorter, is
// fitted to 1.5e-7 of 1 only: off by 0.6% of the value at z = -7, 2% at -10).
__device__ __forceinline__ float tail_of(float z, float* bell) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(fmaf(0.42f, x, 1.f));
  float p = fmaf(t, -0.157329574f, 0.454156995f);
  p = fmaf(t, p, -0.0476845726f);
  p = fmaf(t, p, 0.286179572f);
  p = fmaf(t, p, 0.227307111f);
  p = t * fmaf(t, p, 0.237370476f);
  *bell = __builtin_amdgcn_exp2f(-1.4426950408889634f * x * x);
  return 0.5f * p * *bell;
}

template <int ACT, class T>
__device__ __forceinline__ float act_of(float z) {
  constexpr bool SHORT = sizeof(T) == 2;
  if constexpr (ACT == ACT_RELU) return z < 0.f ? 0.f : z;
  if constexpr (ACT == ACT_GELU) {
    if constexpr (SHORT) {
      float bell;
      const float q = tail_of(z, &bell);
      return z < -1e4f ? 0.f : z * (z < 0.f ? q : 1.f - q);
    }
    return z < -1e4f ? 0.f : 0.5f * z * erfcf(z * -0.70710678118654752f);
  }
  if constexpr (ACT == ACT_SILU) {
    if constexpr (SHORT)
      return z < -1e4f ? 0.f : z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
    return z < -1e4f ? 0.f : z / (1.f + expf(-z));
  }
  return z;
}
template <int ACT, class T>
__device__ __forceinline__ float slope_of(float z) {
  constexpr bool SHORT = sizeof(T) == 2;
  if constexpr (ACT == ACT_RELU) return z <= 0.f ? 0.f : 1.f;
  if constexpr (ACT == ACT_GELU) {
    float phi, bell;
    if constexpr (SHORT) {
      const float q = tail_of(z, &bell);
      phi = z < 0.f ? q : 1.f - q;
    } else {
      bell = expf(-0.5f * z * z);
      phi = 0.5f * erfcf(z * -0.70710678118654752f);
    }
    const float s = fmaf(z * bell, 0.39894228040143268f, phi);
    return z > 1e4f ? 1.f : (z < -1e4f ? 0.f : s);
  }
  if constexpr (ACT == ACT_SILU) {
    float p;
    if constexpr (SHORT) p = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
    else p = 1.f / (1.f + expf(-z));
    const float s = p * (1.f + z * (1.f - p));
    return z > 1e4f ? 1.f : (z < -1e4f ? 0.f : s);
  }
  return 1.f;
}

// A launch over any number of workgroups that 32 bits count: along one
// dimension of a grid HIP takes fewer than 2^32 threads.  Workgroups from
// `blocks` on have to leave.
constexpr uint32_t GRID_X = 1u << 22;
inline dim3 wide_grid(uint64_t blocks, uint32_t z = 1) {
  return dim3((uint32_t)(blocks < GRID_X ? blocks : GRID_X), (uint32_t)((blocks + GRID_X - 1) / GRID_X), z);
}
__device__ __forceinline__ uint32_t block_id() { return blockIdx.y * GRID_X + blockIdx.x; }

template <class V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Whole numbers over the lanes of a wave, all of them active: the scan by DPP
// moves takes a fraction of one by lane exchanges through LDS.
__device__ __forceinline__ uint64_t wave_incl_sum(uint64_t v) {
  v += dpp_take64<0x111, 0xf, 0>(v);
  v += dpp_take64<0x112, 0xf, 0>(v);
  v += dpp_take64<0x114, 0xf, 0>(v);
  v += dpp_take64<0x118, 0xf, 0>(v);
  v += dpp_take64<0x142, 0xa, 0>(v);
  v += dpp_take64<0x143, 0xc, 0>(v);
  uint32_t lo = (uint32_t)v, hi = (uint32_t)(v >> 32);
  asm volatile("" : "+v"(lo), "+v"(hi));
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t wave_total(uint64_t v) { return bcast64(wave_incl_sum(v), 63u); }

// The largest value of a wave (NaN counts as none), in every lane.
__device__ __forceinline__ float wave_top(float v) {
#define TK_STEP(ctrl, rows) \
  v = fmaxf(v, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)0xFF800000u, (int)__float_as_uint(v), ctrl, rows, 0xf, false)))
  TK_STEP(0x111, 0xf);
  TK_STEP(0x112, 0xf);
  TK_STEP(0x114, 0xf);
  TK_STEP(0x118, 0xf);
  TK_STEP(0x142, 0xa);
  TK_STEP(0x143, 0xc);
#undef TK_STEP
  uint32_t u = __float_as_uint(v);
  asm volatile("" : "+v"(u));
  return __uint_as_float(wave_bcast(u, 63u));
}

// Exclusive sums of whole numbers over the threads of a workgroup; *total: of
// all.  `part`: shared, one for each wave; it may be used anew when this returns.
template <uint32_t THREADS, class V>
__device__ __forceinline__ V thread_scan(V v, V* part, V* total) {
  const V up = wave_incl_sum(v);
  if (threadIdx.x % 64 == 63) part[threadIdx.x / 64] = up;
  __syncthreads();
  V before = 0, all = 0;
#pragma unroll
  for (uint32_t w = 0; w < THREADS / 64; ++w) {
    if (w < threadIdx.x / 64) before += part[w];
    all += part[w];
  }
  __syncthreads();
  *total = all;
  return before + up - v;
}

}  // namespace tk
