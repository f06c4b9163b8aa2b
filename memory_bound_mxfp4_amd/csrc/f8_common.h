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
template <typename T>
__device__ __forceinline__ float f8_side(float t, float middle, T beyond) {
  const uint32_t b = __float_as_uint(middle);
  return copysignf(__uint_as_float(beyond > T(0) ? b + 1 : beyond < T(0) ? b - 1 : b), t);
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

// A block's scale, from the bits of its largest magnitude: fp32(amax / 448).  The quotient by
// the constant takes one correction (the same as the division for every significand, as long as
// nothing leaves the normal numbers); its reciprocal only has to be near.
struct F8Scale {
  float stored, inv;
  bool zero;  // all codes 0
  bool tiny;  // a scale whose fp32 reciprocal would overflow, or that is far from amax / 448
};
__device__ __forceinline__ F8Scale f8_scale(uint32_t amax_bits) {
  constexpr float C = 1.0f / kF8Max;
  F8Scale r;
  const bool bad = amax_bits >= 0x7F800000u;
  const float amax = __uint_as_float(amax_bits), near = amax * C;
  float s = fmaf(fmaf(-near, kF8Max, amax), C, near);
  r.tiny = amax < 0x1p-90f;
  if (r.tiny) {
    s = amax / kF8Max;
    asm volatile("" : "+v"(s));  // rare: a branch, and not a division for every block
  }
  r.stored = bad ? __uint_as_float(0x7FC00000u) : s;
  r.zero = bad || s == 0.0f;
  r.inv = __builtin_amdgcn_rcpf(s);
  return r;
}

// 8 elements of a block to codes, each the nearest to the exact quotient x / scale.  x * inv
// is within three of its last places of the quotient (two for the reciprocal, one for the product);
// where that leaves it in doubt, the sign of x - middle * scale decides: a fused multiply-add
// rounds that once, and so keeps its sign and whether it is 0 (its last place is 2^-132 or more).
// Quotients of 16-bit numbers are middles quite often (one in a hundred where the
// block's largest is a multiple of 7), so most waves come through here.  Numbers below
// 2^-6, which some 4% of the waves have of normal values, are tested apart.
__device__ __forceinline__ u32x2 f8_quant8(const float* v, const F8Scale& r) {
  constexpr int TOL = 6;
  float t[8];
  uint32_t doubt = ~0u, least = ~0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = v[i] * r.inv;
    const uint32_t b = __float_as_uint(t[i]);
    doubt = min(doubt, (b << 12) - ((F8_HALF - TOL) << 12));  // the bits rounded away, from just below the middle on
    least = min(least, (b << 1) - 1u);
  }
  if (r.tiny) {
    const double s = (double)r.stored;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t[i] = f8_clamp((float)((double)v[i] / s));
      if (f8_near<TOL>(t[i])) t[i] = f8_side(t[i], f8_middle(t[i]), fma(-(double)f8_middle(t[i]), s, (double)fabsf(v[i])));
    }
  } else if (doubt <= (2u * TOL) << 12 || least < 0x79000000u - 1u) {  // 0x3C800000 is 2^-6
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float m = f8_middle(t[i]), moved = f8_side(t[i], m, fmaf(-m, r.stored, fabsf(v[i])));
      t[i] = f8_near<TOL>(t[i]) ? moved : t[i];
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

// The 8 elements of a row that chunk c stands for; a block is 16 chunks.  VEC: those from 8 c on,
// for rows aligned to 16 bytes whose length is a multiple of 8, in wide accesses; else 16 apart within
// the block, so that the 16 lanes of a block touch neighbours (4096 rows of 4999 fp32 quantised: 33 us, 3.1 TB/s).
template <bool VEC>
__device__ __forceinline__ int element(int c, int i) {
  return VEC ? 8 * c + i : c / kLanes * kBlock + c % kLanes + kLanes * i;
}

// They in fp32, zeros from `end` on.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* row, int c, int end, float* v) {
  if constexpr (VEC) {
    u32x4 d[2] = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
    if (8 * c < end) {
      const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const char*>(row) + (size_t)c * 8 * Elem<DT>::bytes);
      d[0] = p[0];
      if constexpr (Chunk<DT>::N == 4) d[1] = p[1];
    }
    Chunk<DT>::widen(d[0], v);
    if constexpr (Chunk<DT>::N == 4) Chunk<DT>::widen(d[1], v + 4);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = element<VEC>(c, i) < end ? load_f32<DT>(row, element<VEC>(c, i)) : 0.0f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store8_codes(void* row, int c, int end, const u32x2& o) {
  if constexpr (VEC) {
    if (8 * c < end) reinterpret_cast<u32x2*>(row)[c] = o;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (element<VEC>(c, i) < end) static_cast<uint8_t*>(row)[element<VEC>(c, i)] = (uint8_t)(o[i / 4] >> (i % 4 * 8));
  }
}

}  // namespace moe
