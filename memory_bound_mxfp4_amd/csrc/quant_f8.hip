// quant_f8.hip -- rows of activations to e4m3 codes with a scale for each block
// of 128, read once.
#include "f8_common.h"

namespace moe {

// 16 lanes take a block, and U blocks one after another with all their loads in flight; a
// workgroup takes them of 16 rows, so that the scales it writes lie 16 side by side.  Bound by
// memory: 32768 rows of 1536 bf16 33 to 35 us (4.3 to 4.6 TB/s; a large copy has 5.0), of fp32 46 (5.5); 4096 rows
// of 4999 fp32, which no wide load fits, 33 (3.1).
template <int DT, bool VEC, int U>
__global__ __launch_bounds__(256) void k_quant_f8(const void* __restrict__ x, size_t x_stride, int row0, int rows,
                                                  int K, unsigned blocks, unsigned groups, uint8_t* __restrict__ q,
                                                  float* __restrict__ scale) {
  const unsigned b = blockIdx.x % groups * U;
  const size_t row = row0 + (size_t)(blockIdx.x / groups) * 16 + threadIdx.x / kLanes;
  if (row >= (size_t)rows) return;
  const int lane = threadIdx.x % kLanes, c = (int)b * kLanes + lane;
  const char* src = static_cast<const char*>(x) + row * x_stride * Elem<DT>::bytes;
  float v[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) load8<DT, VEC>(src, c + u * kLanes, K, v[u]);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (b + u >= blocks) return;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[u][i]));
    const F8Scale s = f8_scale(block_max_bits(m));
    if (lane == 0) scale[(size_t)(b + u) * rows + row] = s.stored;
    store8_codes<VEC>(q + row * K, c + u * kLanes, K, f8_quant8(v[u], s));
  }
}

template <int DT, bool VEC, int U>
static void quant_launch(const void* x, size_t x_stride, int rows, int K, uint8_t* q, float* scale, hipStream_t s) {
  const unsigned blocks = (K + kBlock - 1) / kBlock, groups = (blocks + U - 1) / U;
  // a launch holds at most 2^31 threads: long calls go in pieces of whole rows
  const size_t most = ((size_t)1 << 31) / 256 / groups * 16, step = most < (size_t)rows ? most : rows;
  for (size_t r0 = 0; r0 < (size_t)rows; r0 += step) {
    const size_t n = rows - r0 < step ? rows - r0 : step;
    hipLaunchKernelGGL((k_quant_f8<DT, VEC, U>), dim3((unsigned)((n + 15) / 16 * groups)), dim3(256), 0, s, x, x_stride,
                       (int)r0, rows, K, blocks, groups, q, scale);
  }
}

template <int DT>
static void quant_dt(const void* x, size_t x_stride, int rows, int K, uint8_t* q, float* scale, hipStream_t s) {
  const bool vec = K % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                   (rows == 1 || x_stride * Elem<DT>::bytes % 16 == 0) && reinterpret_cast<uintptr_t>(q) % 8 == 0;
  // Two blocks a lane where there is work for all CUs (32768 rows of 1536 bf16: 33.0 us for 36.5, four 33.8;
  // 509 rows of 7056 fp16: 5.7 for 5.3).
  const bool two = ((size_t)rows + 15) / 16 * ((K + kBlock - 1) / kBlock) >= 4096;
#define QUANT(VEC, U) quant_launch<DT, VEC, U>(x, x_stride, rows, K, q, scale, s)
  if (vec) two ? QUANT(true, 2) : QUANT(true, 1);
  else two ? QUANT(false, 2) : QUANT(false, 1);
#undef QUANT
}

hipError_t launch_quant_f8(const void* x, int dtype, size_t x_stride, int rows, int K, uint8_t* q, float* scale,
                           hipStream_t s) {
  if (dtype == MOE_DTYPE_BF16) quant_dt<MOE_DTYPE_BF16>(x, x_stride, rows, K, q, scale, s);
  else if (dtype == MOE_DTYPE_F16) quant_dt<MOE_DTYPE_F16>(x, x_stride, rows, K, q, scale, s);
  else quant_dt<MOE_DTYPE_F32>(x, x_stride, rows, K, q, scale, s);
  return hipGetLastError();
}

}  // namespace moe
