// i8_common.h -- device helpers of the routing and 8-bit kernels: loads and
// stores of the three float types, and the exact rounding of a quotient.
// Internal to libmoe_mxfp4.so.
#pragma once

#include <hip/hip_fp16.h>

#include "internal.h"
#include "mx_common.h"

typedef int i32x4 __attribute__((ext_vector_type(4)));

namespace moe {

// Between LDS writes of one lane and reads of another lane of the same wave: orders them
// for the compiler too (the hardware keeps a wave's LDS accesses in order, so this becomes
// no instruction beyond waits that the reads' results need anyway).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

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

// A sum with its two scales, three roundings.  The scales are not multiplied with each
// other first: their product may leave fp32's normal numbers where the result does not (a
// sum of 0 would become NaN, small rows would lose bits).  A sum is a whole number, so
// sum * w_scale, a multiple of the last bit of w_scale, is exact where it is subnormal, and
// as |sum| <= 2^30 it overflows for no w_scale up to 2^97.
__device__ __forceinline__ float scaled(int sum, float x_scale, float w_scale) {
  return (float)sum * w_scale * x_scale;
}

// silu(g) * u with the accurate exponential: the result is within a few fp32
// roundings of the formula for every g and finite u.  Below -80, where exp(-g) may
// overflow although the result does not vanish, 1 + exp(-g) is exp(-g) to fp32 and
// g exp(g) is taken in factors: exp(-80), and twice exp((g + 80) / 2), which is a normal
// number down to -254.  From there on no u leaves more than 0.
__device__ __forceinline__ float swiglu_low(float g, float u) {
  g = fmaxf(g, -300.0f);
  const float t = expf(0.5f * (g + 80.0f));
  return g * 1.8048513878454153e-35f * u * t * t;
}
// Above that.
__device__ __forceinline__ float swiglu_rest(float g, float u) { return g / (1.0f + expf(-g)) * u; }
__device__ __forceinline__ float swiglu_f(float g, float u) { return g < -80.0f ? swiglu_low(g, u) : swiglu_rest(g, u); }

// ---- rows to 8-bit codes ---------------------------------------------------------
//
// scale = fp32(amax / 127), q = the integer nearest to x / scale, ties to even.
// The quotient is rounded as if it were exact: in fp64 x * (1 / scale) is within
// 2^-44 of it, and unless it is the middle between two codes the exact quotient
// is at least 2^-26 away from one (2 x and an odd multiple of the scale are
// multiples of 2^-1 of the scale's last bit where they can be that close).  So a
// first rounding to a multiple of 2^-40 gives the middle exactly where it is one
// and leaves every other value on its side.
__device__ __forceinline__ int quant_code(float x, double inv) {
  const double t = ((double)x * inv + 6144.0) - 6144.0;  // 6144 = 1.5 * 2^12
  return (int)fmin(fmax(rint(t), -127.0), 127.0);
}

// Bits of the largest magnitude: NaN and infinity compare above every finite
// value as integers, so one maximum finds both the scale and a bad row.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t wave_max_bits(uint32_t m) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, WAVE));
  return m;
}

// A row's scale and what its codes are computed with.
struct RowScale {
  float stored, inv;
  double inv64;
  bool zero;  // all codes 0
  bool tiny;  // a scale whose fp32 reciprocal would overflow
};
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
  RowScale r;
  const bool bad = amax_bits >= 0x7F800000u;
  const float s = __uint_as_float(amax_bits) / 127.0f;
  r.stored = bad ? __uint_as_float(0x7FC00000u) : s;
  r.zero = bad || s == 0.0f;
  r.tiny = s < 0x1p-100f;
  r.inv64 = 1.0 / (double)s;
  r.inv = (float)r.inv64;
  return r;
}

// N codes, four to a dword.  x * inv + 1.5 * 2^23 has the nearest integer to
// x * inv in its low bits; where that quotient (off by under 2^-15) is not
// clear of the middle between two codes, the exact rule above decides.
template <int N>
__device__ __forceinline__ void quant_chunk(const float* v, const RowScale& r, uint32_t* out) {
  constexpr float MAGIC = 12582912.0f;
  uint32_t b[N];
  float off = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float t = fmaf(v[i], r.inv, MAGIC);
    b[i] = __float_as_uint(t);
    off = fmaxf(off, fabsf(fmaf(v[i], r.inv, MAGIC - t)));
  }
  if (off > 0.4999f || r.tiny) {
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = (uint32_t)quant_code(v[i], r.inv64);
  }
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const uint32_t lo = __builtin_amdgcn_perm(b[i + 1], b[i], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[i + 3], b[i + 2], 0x0C0C0400u);
    out[i / 4] = r.zero ? 0u : (lo | (hi << 16));
  }
}

}  // namespace moe
