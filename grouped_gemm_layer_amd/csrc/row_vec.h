// 16-byte pieces of rows whose only alignment is that of their elements
// (internal).  Global loads and stores of gfx950 take any byte address, so one
// code path serves aligned rows, odd lengths and odd pitches; the last piece of
// a row, shorter than 16 bytes, goes element by element.
#pragma once

#include "moe_internal.h"

namespace moe {

// fp32 -> bf16 by the conversion instruction: nearest, ties to even; a NaN stays a NaN
__device__ __forceinline__ bf16_t cvt_bf16(float f) { return __builtin_bit_cast(bf16_t, (__bf16)f); }
__device__ __forceinline__ uint32_t cvt_bf16x2(float a, float b) {
  return (uint32_t)cvt_bf16(a) | ((uint32_t)cvt_bf16(b) << 16);
}

typedef uint32_t u32x4v_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4u_t __attribute__((ext_vector_type(4), aligned(2)));   // at any element's address

template <typename T> struct RowVec;

template <typename T>
struct RowVecBase {
  static constexpr int N = 16 / (int)sizeof(T);
  u32x4v_t raw;

  template <bool NT>
  static __device__ __forceinline__ u32x4v_t ld(const T* p, int n) {
    if (n == N) {
      if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const u32x4u_t*>(p));
      else return *reinterpret_cast<const u32x4u_t*>(p);
    }
    u32x4v_t v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 4) v[i] = __builtin_bit_cast(uint32_t, p[i]);
        else v[i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[i]) << (16 * (i % 2));
      }
    return v;
  }
  template <bool NT>
  static __device__ __forceinline__ void st(T* p, int n, u32x4v_t v) {
    if (n == N) {
      if constexpr (NT) __builtin_nontemporal_store((u32x4u_t)v, reinterpret_cast<u32x4u_t*>(p));
      else *reinterpret_cast<u32x4u_t*>(p) = v;
      return;
    }
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 4) {
          const uint32_t w = v[i];   // a value of its own: a bit cast of the vector's element takes element 0
          p[i] = __builtin_bit_cast(T, w);
        }
        else p[i] = (T)(v[i / 2] >> (16 * (i % 2)));
      }
  }
};

template <> struct RowVec<bf16_t> : RowVecBase<bf16_t> {
  static __device__ __forceinline__ RowVec load(const bf16_t* p, int n) { return {ld<false>(p, n)}; }
  static __device__ __forceinline__ RowVec load_once(const bf16_t* p, int n) { return {ld<true>(p, n)}; }
  __device__ __forceinline__ void store(bf16_t* p, int n) const { st<false>(p, n, raw); }
  __device__ __forceinline__ void store_once(bf16_t* p, int n) const { st<true>(p, n, raw); }
  __device__ __forceinline__ void unpack(float (&f)[N]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(raw[i] << 16);
      f[2 * i + 1] = __uint_as_float(raw[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ RowVec pack(const float (&f)[N]) {
    return {u32x4v_t{cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]), cvt_bf16x2(f[6], f[7])}};
  }
};

template <> struct RowVec<float> : RowVecBase<float> {
  static __device__ __forceinline__ RowVec load(const float* p, int n) { return {ld<false>(p, n)}; }
  static __device__ __forceinline__ RowVec load_once(const float* p, int n) { return {ld<true>(p, n)}; }
  __device__ __forceinline__ void store(float* p, int n) const { st<false>(p, n, raw); }
  __device__ __forceinline__ void store_once(float* p, int n) const { st<true>(p, n, raw); }
  __device__ __forceinline__ void unpack(float (&f)[N]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(raw[i]);
  }
  static __device__ __forceinline__ RowVec pack(const float (&f)[N]) {
    return {u32x4v_t{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])}};
  }
};

// Sum over the 64 lanes of a wave, the same value in every lane (DPP steps
// inside rows of 16, then the two row swaps).
__device__ __forceinline__ float wave_sum(float v) {
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));    // quad_perm 1,0,3,2
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false));    // quad_perm 2,3,0,1
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false));   // row_half_mirror
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false));   // row_mirror
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

}  // namespace moe
