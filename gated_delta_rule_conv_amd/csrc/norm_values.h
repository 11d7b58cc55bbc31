// Values of any alignment as fp32 vectors of 4, sums over lanes, and the range of a sum of squares: what the
// norm kernels share.
#pragma once

#include "device_common.h"

namespace gdn {

// 4 values as fp32 from an address aligned to the element only
typedef float uf32x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t uu16x4 __attribute__((ext_vector_type(4), aligned(2)));

template <typename T>
__device__ __forceinline__ float get(const T* p) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(*p);
  else return *p;
}

// (the hardware conversion: nearest even, and a NaN of any payload stays one)
__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)); }

template <typename T>
__device__ __forceinline__ void put(T* p, float v) {
  if constexpr (sizeof(T) == 2) *p = to_bf16(v);
  else *p = v;
}

// values [k, k + 4) of a group of `size`, zeros past its end
template <typename T>
__device__ __forceinline__ f32x4 load4u(const T* p, int k, int size) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (k + 3 < size) {
    if constexpr (sizeof(T) == 2) {
      const uu16x4 r = *reinterpret_cast<const uu16x4*>(p + k);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = bf16_to_f32(r[e]);
    } else {
      const uf32x4 r = *reinterpret_cast<const uf32x4*>(p + k);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = r[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (k + e < size) v[e] = get(p + k + e);
  }
  return v;
}

template <typename T>
__device__ __forceinline__ void store4u(T* p, int k, int size, const f32x4& v) {
  if (k + 3 < size) {
    if constexpr (sizeof(T) == 2) {
      uu16x4 r;
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = to_bf16(v[e]);
      *reinterpret_cast<uu16x4*>(p + k) = r;
    } else {
      uf32x4 r;
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = v[e];
      *reinterpret_cast<uf32x4*>(p + k) = r;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (k + e < size) put(p + k + e, v[e]);
  }
}

__device__ __forceinline__ f32x4 load_any(const void* p, int bf16, int64_t off, int k, int size) {
  return bf16 ? load4u(static_cast<const uint16_t*>(p) + off, k, size)
              : load4u(static_cast<const float*>(p) + off, k, size);
}

// a lane's V vectors of a group
template <int LPG, int V>
__device__ __forceinline__ void load_all(const void* p, int bf16, int64_t off, int c, int size, f32x4 (&v)[V]) {
  if (bf16) {
#pragma unroll
    for (int t = 0; t < V; ++t) v[t] = load4u(static_cast<const uint16_t*>(p) + off, 4 * (c + LPG * t), size);
  } else {
#pragma unroll
    for (int t = 0; t < V; ++t) v[t] = load4u(static_cast<const float*>(p) + off, 4 * (c + LPG * t), size);
  }
}

// Sum over aligned groups of L lanes, the last two steps by gfx950's swaps of lane rows.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  v = group_sum<(L < 16 ? L : 16)>(v);
  if constexpr (L >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if constexpr (L >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  return v;
}

// Squares leave the fp32 range long before values do. Where the mean square is not a number well inside it
// (overflow, underflow, an infinity in the group), the group is taken again times 2^range_shift, which puts the
// larger of its largest magnitude and sqrt(eps) near 1. Only such groups pay: 15717 x 32 x 128 fp32 values take 94 us
// with the test and without.
__device__ __forceinline__ bool in_range(float ms) { return ms > 0x1p-100f && ms < __builtin_inff(); }
__device__ __forceinline__ int range_shift(float most, float eps) {
  if (!(most < __builtin_inff())) return 0;
  const int e = (__builtin_amdgcn_frexp_expf(eps) + 1) >> 1;
  if (most == 0.f) return eps > 0.f ? -e : 0;
  const int m = __builtin_amdgcn_frexp_expf(most);
  return eps > 0.f && e > m ? -e : -m;
}
__device__ __forceinline__ float largest(const f32x4& v) {
  return fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
}

}  // namespace gdn
