// quant.hip -- rows of activations to 8-bit codes with one scale each, read
// once: bound by memory (8192 rows of 7168 bf16: 33 us, 5.3 TB/s; 37 rows: 3.8 us,
// latency).
#include "i8_common.h"

namespace moe {

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
    q[row * K + i] = rs.zero ? (int8_t)0 : (int8_t)quant_code(load_f32<DT>(x, row * x_stride + i), rs.inv64);
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
