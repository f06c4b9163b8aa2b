// i8_common.h -- device helpers of the routing and 8-bit kernels: loads and
// stores of the three float types, and the exact rounding of a quotient.
// Internal to libmoe_mxfp4.so.
#pragma once

#include <hip/hip_fp16.h>

#include "internal.h"
#include "mx_common.h"

typedef int i32x4 __attribute__((ext_vector_type(4)));

namespace moe {

// Element i of a bf16, fp16 or fp32 array, widened to fp32 (exact).
template <int DT>
__device__ __forceinline__ float load_f32(const void* p, size_t i) {
  if constexpr (DT == MOE_DTYPE_BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  else if constexpr (DT == MOE_DTYPE_F16) return __half2float(static_cast<const __half*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

template <int DT>
struct Elem;
template <>
struct Elem<MOE_DTYPE_BF16> {
  static constexpr int bytes = 2;
};
template <>
struct Elem<MOE_DTYPE_F16> {
  static constexpr int bytes = 2;
};
template <>
struct Elem<MOE_DTYPE_F32> {
  static constexpr int bytes = 4;
};

// 16 bytes of a row: 8 elements of 2 bytes or 4 of 4.
template <int DT>
struct Chunk {
  static constexpr int N = 16 / Elem<DT>::bytes;
  static __device__ __forceinline__ void widen(const u32x4& c, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == MOE_DTYPE_BF16) {
        v[2 * i] = bf16_lo(c[i]);
        v[2 * i + 1] = bf16_hi(c[i]);
      } else if constexpr (DT == MOE_DTYPE_F16) {
        v[2 * i] = __half2float(__ushort_as_half((uint16_t)c[i]));
        v[2 * i + 1] = __half2float(__ushort_as_half((uint16_t)(c[i] >> 16)));
      } else {
        v[i] = __uint_as_float(c[i]);
      }
    }
  }
};

__device__ __forceinline__ uint16_t f32_to_f16(float f) { return __half_as_ushort(__float2half(f)); }

// Two values rounded to nearest even and packed, the first one low.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == MOE_DTYPE_BF16) {
    bf16x2 h;
    h[0] = (__bf16)a;
    h[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, h);
  } else {
    return (uint32_t)f32_to_f16(a) | ((uint32_t)f32_to_f16(b) << 16);
  }
}

__device__ __forceinline__ void store_y(void* y, int dtype, size_t i, float v) {
  if (dtype == MOE_DTYPE_BF16) static_cast<uint16_t*>(y)[i] = f32_to_bf16(v);
  else if (dtype == MOE_DTYPE_F16) static_cast<uint16_t*>(y)[i] = f32_to_f16(v);
  else static_cast<float*>(y)[i] = v;
}

// silu(g) * u with the accurate exponential: the result is within a few fp32
// roundings of the formula for every finite g (exp overflows to inf and the
// quotient to -0 for very negative g).
__device__ __forceinline__ float swiglu_f(float g, float u) { return g / (1.0f + expf(-g)) * u; }

}  // namespace moe
