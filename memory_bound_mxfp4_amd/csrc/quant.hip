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

__device__ __forceinline__ uint32_t wave_max_bits(uint32_t m) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, WAVE));
  return m;
}

// A row's scale and what its codes are computed with.
struct RowScale {
  float stored, s, inv, up;  // up: power of two that lifts a scale whose reciprocal would overflow
  bool zero;                 // all codes 0
};
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
  RowScale r;
  const bool bad = amax_bits >= 0x7F800000u;
  const float s = __uint_as_float(amax_bits) / 127.0f;
  r.stored = bad ? __uint_as_float(0x7FC00000u) : s;
  r.zero = bad || s == 0.0f;
  r.up = s < 0x1p-100f ? 0x1p64f : 1.0f;
  r.s = s * r.up;
  r.inv = 1.0f / r.s;
  return r;
}

// Any stride, any alignment: element by element, the row read twice.
template <int DT>
__global__ __launch_bounds__(256) void k_quant_rows_any(const void* __restrict__ x, size_t x_stride, int K,
                                                        int8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ uint32_t part[4];
  const size_t row = blockIdx.x;
  uint32_t m = 0;
  for (int i = threadIdx.x; i < K; i += 256) m = max(m, abs_bits(load_f32<DT>(x, row * x_stride + i)));
  m = wave_max_bits(m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  const RowScale rs = row_scale(max(max(part[0], part[1]), max(part[2], part[3])));
  if (threadIdx.x == 0) scale[row] = rs.stored;
  for (int i = threadIdx.x; i < K; i += 256)
    q[row * K + i] = rs.zero ? (int8_t)0 : (int8_t)quant_code(load_f32<DT>(x, row * x_stride + i) * rs.up, rs.s, rs.inv);
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
  if (off > 0.4999f || r.up != 1.0f) {
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = (uint32_t)quant_code(v[i] * r.up, r.s, r.inv);
  }
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const uint32_t lo = __builtin_amdgcn_perm(b[i + 1], b[i], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[i + 3], b[i + 2], 0x0C0C0400u);
    out[i / 4] = r.zero ? 0u : (lo | (hi << 16));
  }
}

// Aligned rows of at most NC 16-byte chunks a thread: a row is read once, all
// of its chunks requested before the maximum is taken, and stays in
// registers.  T threads a row (64: a wave, four rows to a workgroup).
template <int DT, int T, int NC>
__global__ __launch_bounds__(256) void k_quant_rows(const u32x4* __restrict__ x, size_t row_chunks, int rows, int C,
                                                    uint32_t* __restrict__ q, float* __restrict__ scale) {
  constexpr int N = Chunk<DT>::N;
  const int tid = threadIdx.x % T;
  const size_t row = (size_t)blockIdx.x * (256 / T) + threadIdx.x / T;
  if (T == 64 && row >= (size_t)rows) return;
  const u32x4* src = x + row * row_chunks;
  u32x4 c[NC];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NC; ++i) c[i] = tid + T * i < C ? src[tid + T * i] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    float v[N];
    Chunk<DT>::widen(c[i], v);
#pragma unroll
    for (int j = 0; j < N; ++j) m = max(m, abs_bits(v[j]));
  }
  m = wave_max_bits(m);
  if constexpr (T == 256) {
    __shared__ uint32_t part[4];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    m = max(max(part[0], part[1]), max(part[2], part[3]));
  }
  const RowScale rs = row_scale(m);
  if (tid == 0) scale[row] = rs.stored;
  uint32_t* dst = q + row * C * (N / 4);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int at = tid + T * i;
    if (at >= C) continue;
    float v[N];
    Chunk<DT>::widen(c[i], v);
    uint32_t o[N / 4];
    quant_chunk<N>(v, rs, o);
    if constexpr (N == 8) reinterpret_cast<u32x2*>(dst)[at] = u32x2{o[0], o[1]};
    else dst[at] = o[0];
  }
}

template <int DT>
static void quant_dt(const void* x, size_t x_stride, int rows, int K, int8_t* q, float* scale, hipStream_t s) {
  constexpr int N = Chunk<DT>::N, ES = Elem<DT>::bytes;
  const int C = K / N;
  const bool whole = K % N == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 && (rows == 1 || x_stride * ES % 16 == 0) &&
                     reinterpret_cast<uintptr_t>(q) % N == 0;
  const size_t rc = x_stride * ES / 16;
  const u32x4* xv = static_cast<const u32x4*>(x);
  uint32_t* qv = reinterpret_cast<uint32_t*>(q);
  const dim3 block(256), waves((rows + 3) / 4);
#define QUANT(T, NC, grid) \
  hipLaunchKernelGGL((k_quant_rows<DT, T, NC>), grid, block, 0, s, xv, rc, rows, C, qv, scale)
  if (!whole || C > 256 * 8)
    hipLaunchKernelGGL(k_quant_rows_any<DT>, dim3(rows), block, 0, s, x, x_stride, K, q, scale);
  else if (C <= 64) QUANT(64, 1, waves);
  else if (C <= 128 && rows > 256) QUANT(64, 2, waves);
  else if (C <= 256 && rows > 256) QUANT(64, 4, waves);
  else if (C <= 256) QUANT(256, 1, dim3(rows));
  else if (C <= 512) QUANT(256, 2, dim3(rows));
  else if (C <= 1024) QUANT(256, 4, dim3(rows));
  else QUANT(256, 8, dim3(rows));
#undef QUANT
}

hipError_t launch_quant_rows(const void* x, int dtype, size_t x_stride, int rows, int K, int8_t* q, float* scale,
                             hipStream_t s) {
  if (dtype == MOE_DTYPE_BF16) quant_dt<MOE_DTYPE_BF16>(x, x_stride, rows, K, q, scale, s);
  else if (dtype == MOE_DTYPE_F16) quant_dt<MOE_DTYPE_F16>(x, x_stride, rows, K, q, scale, s);
  else quant_dt<MOE_DTYPE_F32>(x, x_stride, rows, K, q, scale, s);
  return hipGetLastError();
}

}  // namespace moe
