// f8_common.h -- rows to e4m3 codes with a scale for each block of 128: the
// scale of a block and the exact rounding of a quotient.
// Internal to libmoe_mxfp4.so.
#pragma once

#include "i8_common.h"

namespace moe {

constexpr int kBlock = 128;        // elements of K, and rows of a matrix, that share a scale
constexpr float kF8Max = 448.0f;   // the largest e4m3 number
constexpr int kLanes = kBlock / 8;  // lanes that hold a block, 8 elements each

// Rounding to e4m3 keeps 3 bits behind the leading one, and steps of 2^-9 below 2^-6.  With
// 2^-6 added, a number below 2^-6 has its step at the same place of the significand as the
// numbers up to 2^-5, so one mask finds the bits that are rounded away: the number is the
// middle between two codes where they are exactly F8_HALF.
constexpr uint32_t F8_REST = 0xFFFFFu, F8_HALF = 0x80000u;
__device__ __forceinline__ uint32_t f8_place(float a) { return __float_as_uint(a < 0x1p-6f ? a + 0x1p-6f : a); }

// Whether |t| is within TOL of its last places of a middle.
template <int TOL>
__device__ __forceinline__ bool f8_near(float t) {
  return (f8_place(fabsf(t)) & F8_REST) - (F8_HALF - TOL) <= 2u * TOL;
}

// For t near a middle: that middle, moved to the side that `beyond` names (the sign of what
// the exact quotient is past it; 0: it is the middle, and the conversion's rule for ties holds).
__device__ __forceinline__ float f8_middle(float t) {
  const float a = fabsf(t);
  const float m = __uint_as_float((f8_place(a) & ~F8_REST) | F8_HALF);
  return a < 0x1p-6f ? m - 0x1p-6f : m;
}
__device__ __forceinline__ float f8_side(float t, float middle, double beyond) {
  const uint32_t b = __float_as_uint(middle);
  return copysignf(__uint_as_float(beyond > 0.0 ? b + 1 : beyond < 0.0 ? b - 1 : b), t);
}

// Two numbers within +-448 to codes, in the low or high half of a dword.
template <bool HIGH>
__device__ __forceinline__ uint32_t f8_pair(float a, float b, uint32_t old) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, HIGH);
}
__device__ __forceinline__ float f8_clamp(float t) { return fminf(fmaxf(t, -kF8Max), kF8Max); }

// 8 numbers to 8 codes.
__device__ __forceinline__ u32x2 f8_pack(const float* t) {
  u32x2 o;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    o[i] = f8_pair<true>(t[4 * i + 2], t[4 * i + 3], f8_pair<false>(t[4 * i], t[4 * i + 1], 0u));
  return o;
}

// A block's scale, from the bits of its largest magnitude.
struct F8Scale {
  float stored, inv;
  bool zero;  // all codes 0
  bool tiny;  // a scale whose fp32 reciprocal would overflow, or that is far from amax / 448
};
__device__ __forceinline__ F8Scale f8_scale(uint32_t amax_bits) {
  F8Scale r;
  const bool bad = amax_bits >= 0x7F800000u;
  const float s = __uint_as_float(amax_bits) / kF8Max;
  r.stored = bad ? __uint_as_float(0x7FC00000u) : s;
  r.zero = bad || s == 0.0f;
  r.tiny = s < 0x1p-100f;
  r.inv = 1.0f / s;
  return r;
}

// 8 elements of a block to codes, each the nearest to the exact quotient x / scale.  x * inv
// is within two of its last places of the quotient (half of one for the reciprocal, half
// for the product, twice that where the leading bits differ); where that leaves
// it in doubt, the sign of x - middle * scale decides, which 64 bits hold exactly
// (24 + 5 bits).
__device__ __forceinline__ u32x2 f8_quant8(const float* v, const F8Scale& r) {
  float t[8];
  bool near = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = v[i] * r.inv;
    near |= f8_near<4>(t[i]);
  }
  if (near || r.tiny) {
    const double s = (double)r.stored;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r.tiny) t[i] = f8_clamp((float)((double)v[i] / s));
      if (f8_near<4>(t[i])) {
        const float m = f8_middle(t[i]);
        t[i] = f8_side(t[i], m, fma(-(double)m, s, (double)fabsf(v[i])));
      }
    }
  }
  const u32x2 o = f8_pack(t);
  return r.zero ? u32x2{0u, 0u} : o;
}

// The largest over the 16 lanes that hold a block, in all of them (rotations within 16 lanes).
__device__ __forceinline__ uint32_t block_max_bits(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x122, 0xF, 0xF, false));
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x121, 0xF, 0xF, false));
}

// 8 elements of a row from `at` on, fp32; VEC: aligned to 16 bytes and inside the row,
// else element by element, zeros from `end` on.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* row, int at, int end, float* v) {
  if constexpr (VEC) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const char*>(row) + (size_t)at * Elem<DT>::bytes);
    Chunk<DT>::widen(p[0], v);
    if constexpr (Chunk<DT>::N == 4) Chunk<DT>::widen(p[1], v + 4);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = at + i < end ? load_f32<DT>(row, at + i) : 0.0f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store8_codes(void* row, int at, int end, const u32x2& o) {
  if constexpr (VEC) {
    *reinterpret_cast<u32x2*>(static_cast<char*>(row) + at) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at + i < end) static_cast<uint8_t*>(row)[at + i] = (uint8_t)(o[i / 4] >> (i % 4 * 8));
  }
}

}  // namespace moe
