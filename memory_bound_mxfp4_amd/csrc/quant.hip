// quant.hip -- rows of activations to 8-bit codes with one scale each.
//
// scale = fp32(amax / 127), q = the integer nearest to x / scale.  The
// quotient is rounded as if it were exact: x * (1 / scale) in fp32 is within
// one unit of it, and x - q * scale, one fused multiply-add, is exact there
// (both terms are multiples of 2^-25 of the scale's binade and the
// difference stays under one scale), so comparing twice that remainder with
// the scale decides which side of the middle between two codes x is on.
#include "i8_common.h"

namespace moe {

__device__ __forceinline__ int quant_code(float x, float s, float inv) {
  float q = rintf(x * inv);
  const float r = fmaf(-q, s, x), twice = 2.0f * fabsf(r);
  // past the middle, or on it with an odd code (ties go to the even one)
  if (twice > s || (twice == s && ((int)q & 1))) q += r > 0.0f ? 1.0f : -1.0f;
  return (int)fminf(fmaxf(q, -127.0f), 127.0f);
}

// Bits of the largest magnitude: NaN and infinity compare above every finite
// value as integers, so one maximum finds both the scale and a bad row.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

template <int DT>
__global__ __launch_bounds__(256) void k_quant_rows(const void* __restrict__ x, size_t x_stride, int K,
                                                    int8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ uint32_t part[4];
  const size_t row = blockIdx.x;
  uint32_t m = 0;
  for (int i = threadIdx.x; i < K; i += 256) m = max(m, abs_bits(load_f32<DT>(x, row * x_stride + i)));
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, WAVE));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(part[0], part[1]), max(part[2], part[3]));
  const bool bad = m >= 0x7F800000u;
  const float s = __uint_as_float(m) / 127.0f;
  if (threadIdx.x == 0) scale[row] = bad ? __uint_as_float(0x7FC00000u) : s;
  // a scale too small for its reciprocal: both sides times 2^64, exactly
  const float up = s < 0x1p-100f ? 0x1p64f : 1.0f, su = s * up, inv = 1.0f / su;
  const bool zero = bad || s == 0.0f;
  for (int i = threadIdx.x; i < K; i += 256)
    q[row * K + i] = zero ? (int8_t)0 : (int8_t)quant_code(load_f32<DT>(x, row * x_stride + i) * up, su, inv);
}

hipError_t launch_quant_rows(const void* x, int dtype, size_t x_stride, int rows, int K, int8_t* q, float* scale,
                             hipStream_t s) {
  if (dtype == MOE_DTYPE_BF16)
    hipLaunchKernelGGL(k_quant_rows<MOE_DTYPE_BF16>, dim3(rows), dim3(256), 0, s, x, x_stride, K, q, scale);
  else if (dtype == MOE_DTYPE_F16)
    hipLaunchKernelGGL(k_quant_rows<MOE_DTYPE_F16>, dim3(rows), dim3(256), 0, s, x, x_stride, K, q, scale);
  else
    hipLaunchKernelGGL(k_quant_rows<MOE_DTYPE_F32>, dim3(rows), dim3(256), 0, s, x, x_stride, K, q, scale);
  return hipGetLastError();
}

}  // namespace moe
