// Element types and cache addressing shared by the serving kernels
// (kv_append.hip, attn_prefix.hip, f8b128.hip); gfx950 only.
#pragma once

#include "lqmm_device.hpp"

namespace lqmm {

typedef __bf16 bhalf_t;
typedef __bf16 bhalf8_t __attribute__((ext_vector_type(8)));

struct TypeF32 {
  typedef float elem;
  static constexpr int kBytes = 4;
  static __device__ __forceinline__ void unpack8(const u32x4 (&r)[2], float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = r[i >> 2][i & 3];
      x[i] = __builtin_bit_cast(float, w);
    }
  }
};

struct TypeF16 {
  typedef half_t elem;
  typedef half8_t vec8;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float4_t mfma16(vec8 a, vec8 b, float4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ float16_t mfma32(vec8 a, vec8 b, float16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};

struct TypeBF16 {
  typedef bhalf_t elem;
  typedef bhalf8_t vec8;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float4_t mfma16(vec8 a, vec8 b, float4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ float16_t mfma32(vec8 a, vec8 b, float16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};

// Eight consecutive elements at p (16-byte aligned) as fp32.
template <class T>
__device__ __forceinline__ void load8(const typename T::elem *p, float (&x)[8]) {
  if constexpr (T::kBytes == 4) {
    const u32x4 r[2] = {*reinterpret_cast<const u32x4 *>(p), *reinterpret_cast<const u32x4 *>(p + 4)};
    TypeF32::unpack8(r, x);
  } else {
    const typename T::vec8 v = *reinterpret_cast<const typename T::vec8 *>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
  }
}

// Eight fp32 values rounded (nearest even) and stored at p (16-byte aligned).
template <class T>
__device__ __forceinline__ void store8(typename T::elem *p, const float (&x)[8]) {
  typename T::vec8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (typename T::elem)x[i];
  *reinterpret_cast<typename T::vec8 *>(p) = v;
}

// Largest or summed value over the four 16-lane groups of a wave, in every
// lane (v_permlane32_swap / v_permlane16_swap exchange half-waves and rows).
__device__ __forceinline__ float max_over_rows(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t a0 = a[0], a1 = a[1];
  const float m = fmaxf(__builtin_bit_cast(float, a0), __builtin_bit_cast(float, a1));
  const uint32_t w = __builtin_bit_cast(uint32_t, m);
  const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  const uint32_t b0 = b[0], b1 = b[1];
  return fmaxf(__builtin_bit_cast(float, b0), __builtin_bit_cast(float, b1));
}
__device__ __forceinline__ float sum_over_rows(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t a0 = a[0], a1 = a[1];
  const float m = __builtin_bit_cast(float, a0) + __builtin_bit_cast(float, a1);
  const uint32_t w = __builtin_bit_cast(uint32_t, m);
  const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  const uint32_t b0 = b[0], b1 = b[1];
  return __builtin_bit_cast(float, b0) + __builtin_bit_cast(float, b1);
}

// The same over the two half-waves.
__device__ __forceinline__ float max_over_halves(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t a0 = a[0], a1 = a[1];
  return fmaxf(__builtin_bit_cast(float, a0), __builtin_bit_cast(float, a1));
}
__device__ __forceinline__ float sum_over_halves(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t a0 = a[0], a1 = a[1];
  return __builtin_bit_cast(float, a0) + __builtin_bit_cast(float, a1);
}

// Waits until at most N of this wave's memory loads are out and its LDS
// operations are done, then joins the workgroup barrier.
template <int N>
__device__ __forceinline__ void wait_loads_and_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// BYTES (4 or 16) of each lane from src to LDS: lane i's go to dst + BYTES * i
// (dst is the same in all lanes).
typedef __attribute__((address_space(1))) const void *global_ptr;
typedef __attribute__((address_space(3))) void *lds_ptr;
template <int BYTES>
__device__ __forceinline__ void load_to_lds(const void *src, uint8_t *dst) {
  static_assert(BYTES == 4 || BYTES == 16, "load size");
  if constexpr (BYTES == 16)
    __builtin_amdgcn_global_load_lds((global_ptr)(uintptr_t)src, (lds_ptr)dst, 16, 0, 0);
  else
    __builtin_amdgcn_global_load_lds((global_ptr)(uintptr_t)src, (lds_ptr)dst, 4, 0, 0);
}

}  // namespace lqmm
