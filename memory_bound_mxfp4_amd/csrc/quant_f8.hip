// quant_f8.hip -- rows of activations to e4m3 codes with a scale for each block
// of 128, read once.
#include "f8_common.h"

namespace moe {

// 16 lanes take a block; a workgroup takes one block of each of 16 rows, so that the
// 16 scales it writes lie side by side.
template <int DT, bool VEC>
__global__ __launch_bounds__(256) void k_quant_f8(const void* __restrict__ x, size_t x_stride, int row0, int rows,
                                                  int K, unsigned blocks, uint8_t* __restrict__ q,
                                                  float* __restrict__ scale) {
  const unsigned b = blockIdx.x % blocks;
  const size_t row = row0 + (size_t)(blockIdx.x / blocks) * 16 + threadIdx.x / kLanes;
  if (row >= (size_t)rows) return;
  const int lane = threadIdx.x % kLanes, at = (int)b * kBlock + 8 * lane;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const bool any = at < K;
  if (any) load8<DT, VEC>(static_cast<const char*>(x) + row * x_stride * Elem<DT>::bytes, at, K, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
  const F8Scale s = f8_scale(block_max_bits(m));
  if (lane == 0) scale[(size_t)b * rows + row] = s.stored;
  if (any) store8_codes<VEC>(q + row * K, at, K, f8_quant8(v, s));
}

template <int DT>
static void quant_dt(const void* x, size_t x_stride, int rows, int K, uint8_t* q, float* scale, hipStream_t s) {
  const bool vec = K % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                   (rows == 1 || x_stride * Elem<DT>::bytes % 16 == 0) && reinterpret_cast<uintptr_t>(q) % 8 == 0;
  const unsigned blocks = (K + kBlock - 1) / kBlock;
  // a launch holds at most 2^31 threads: long calls go in pieces of whole rows
  const int step = (int)((((size_t)1 << 31) / 256 / blocks) * 16 < (size_t)rows ? (((size_t)1 << 31) / 256 / blocks) * 16 : rows);
  for (size_t r0 = 0; r0 < (size_t)rows; r0 += step) {
    const size_t n = rows - r0 < (size_t)step ? rows - r0 : step;
    const dim3 grid((unsigned)((n + 15) / 16 * blocks)), block(256);
    if (vec) hipLaunchKernelGGL((k_quant_f8<DT, true>), grid, block, 0, s, x, x_stride, (int)r0, rows, K, blocks, q, scale);
    else hipLaunchKernelGGL((k_quant_f8<DT, false>), grid, block, 0, s, x, x_stride, (int)r0, rows, K, blocks, q, scale);
  }
}

hipError_t launch_quant_f8(const void* x, int dtype, size_t x_stride, int rows, int K, uint8_t* q, float* scale,
                           hipStream_t s) {
  if (dtype == MOE_DTYPE_BF16) quant_dt<MOE_DTYPE_BF16>(x, x_stride, rows, K, q, scale, s);
  else if (dtype == MOE_DTYPE_F16) quant_dt<MOE_DTYPE_F16>(x, x_stride, rows, K, q, scale, s);
  else quant_dt<MOE_DTYPE_F32>(x, x_stride, rows, K, q, scale, s);
  return hipGetLastError();
}

}  // namespace moe
