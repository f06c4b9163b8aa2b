// gemm_f8.hip -- the 8-bit floating-point products with a scale for each block
// of 128: y = sum over blocks b of (x_scale[b] * w_scale[b]) * (xq wq^T)_b, for
// one matrix or for the rows of each expert, with SwiGLU on pairs of matrices.
#include "f8_common.h"
#include "tile_device.h"
#include "tile_order.h"

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

namespace moe {

// 16 codes to fp16, which holds every e4m3 number.
struct Wide16 {
  f16x8 h[2];
};
__device__ __forceinline__ Wide16 widen(const i32x4& c) {
  Wide16 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], 1.0f, true);
    o.h[i / 2][i % 2 * 4] = a[0];
    o.h[i / 2][i % 2 * 4 + 1] = a[1];
    o.h[i / 2][i % 2 * 4 + 2] = b[0];
    o.h[i / 2][i % 2 * 4 + 3] = b[1];
  }
  return o;
}

// The products of one block: 16 matrix rows by 16 rows of x over 128 codes of K, summed in
// fp32.  Both operands hold the same 32 codes of K in a lane, so their order within the
// block does not matter.  (The matrix units' own 8-bit products are twice as fast, but align the
// products of 8 neighbouring codes to the largest of them and cut off what is below 2^-13 of it.)
__device__ __forceinline__ f32x4 mfma_block(const i32x4 (&w)[2], const i32x4 (&x)[2]) {
  f32x4 c{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const Wide16 a = widen(w[h]), b = widen(x[h]);
#pragma unroll
    for (int i = 0; i < 2; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.h[i], b.h[i], c, 0, 0, 0);
  }
  return c;
}

constexpr size_t kMaxGroups = ((size_t)1 << 31) / 512;  // workgroups of a launch: its threads, and numbers in int

// 64 rows of x by 64 matrix rows a workgroup of 2 x 2 waves; a block of K at a time through
// one buffer in LDS.
template <int P>
__global__ __launch_bounds__(256) void k_f8_simple(F8Args a, int tiles_n) {
  constexpr int LD = KS + 16;  // rows apart by 36 banks
  __shared__ __attribute__((aligned(16))) int8_t lx[64 * LD], lw[64 * LD];
  __shared__ int yr[64];
  Tile t;
  if (!find_tile<64>(a, blockIdx.x / tiles_n, t)) return;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4, wv = threadIdx.x >> 6, wm = wv & 1, wn = wv >> 1;
  const int i0 = blockIdx.x % tiles_n * (64 / P), K = a.k, kb = (K + kBlock - 1) / kBlock, nb = (a.n + kBlock - 1) / kBlock;
  if (t.e >= a.num_experts) {  // slots without an expert: rows of zeros
    for (int i = threadIdx.x; i < t.rows * (64 / P); i += 256)
      if (i0 + i % (64 / P) < a.n) store_y(a.y, a.y_dtype, (size_t)y_row(a, t.p0 + i / (64 / P)) * a.n + i0 + i % (64 / P), 0.0f);
    return;
  }
  if (threadIdx.x < 64) yr[threadIdx.x] = y_row(a, t.p0 + min((int)threadIdx.x, t.rows - 1));
  __syncthreads();
  f32x4 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int b = 0; b < kb; ++b) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = threadIdx.x + 256 * i, row = c / 8, k = b * KS + c % 8 * 16;
      const int p = P == 2 ? row / 16 % 2 : 0, n = min(i0 + (P == 2 ? row / 32 * 16 + row % 16 : row), a.n - 1);
      i32x4 vx{0, 0, 0, 0}, vw{0, 0, 0, 0};
      if (k < K) {
        vx = *reinterpret_cast<const i32x4*>(a.x + (size_t)x_row(a, yr[row]) * a.x_stride + k);
        vw = *reinterpret_cast<const i32x4*>(a.w + (((size_t)t.e * P + p) * a.n + n) * K + k);
      }
      *reinterpret_cast<i32x4*>(lx + row * LD + c % 8 * 16) = vx;
      *reinterpret_cast<i32x4*>(lw + row * LD + c % 8 * 16) = vw;
    }
    __syncthreads();
    i32x4 fx[2][2], fw[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        fx[i][h] = *reinterpret_cast<const i32x4*>(lx + (16 * (2 * wm + i) + r) * LD + 16 * (4 * h + q));
        fw[i][h] = *reinterpret_cast<const i32x4*>(lw + (16 * (2 * wn + i) + r) * LD + 16 * (4 * h + q));
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float sx = a.x_scale[(size_t)b * a.x_rows + x_row(a, yr[16 * (2 * wm + i) + r])];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float s = sx * a.w_scale[(((size_t)t.e * P + (P == 2 ? j : 0)) * nb + i0 / kBlock) * kb + b];
        const f32x4 v = mfma_block(fw[j], fx[i]);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][j][c] = fmaf(s, v[c], acc[i][j][c]);
      }
    }
    __syncthreads();
  }
  // register c of lane 16 q + r: matrix row 4 q + c of the fragment, row r of x
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = 16 * (2 * wm + i) + r;
    if (m >= t.rows) continue;
#pragma unroll
    for (int j = 0; j < 2 / P; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int n = i0 + (P == 2 ? 16 * wn : 16 * (2 * wn + j)) + 4 * q + c;
        const float v = P == 2 ? swiglu_f(acc[i][0][c], acc[i][1][c]) : acc[i][j][c];
        if (n < a.n) store_y(a.y, a.y_dtype, (size_t)yr[m] * a.n + n, v);
      }
  }
}

F8Plan f8_plan(int, int, bool, int, int, bool) { return F8Plan{0, 64}; }

bool f8_launchable(const F8Plan&, int n, bool swiglu, int max_tiles) {
  return ((size_t)n * (swiglu ? 2 : 1) + 63) / 64 * max_tiles < kMaxGroups;
}

hipError_t launch_gemm_f8(const F8Args& a, const F8Plan&, int max_tiles, hipStream_t s) {
  const int tiles_n = (a.n * (a.swiglu ? 2 : 1) + 63) / 64;
  if (a.swiglu) hipLaunchKernelGGL(k_f8_simple<2>, dim3(tiles_n * max_tiles), dim3(256), 0, s, a, tiles_n);
  else hipLaunchKernelGGL(k_f8_simple<1>, dim3(tiles_n * max_tiles), dim3(256), 0, s, a, tiles_n);
  return hipGetLastError();
}

}  // namespace moe
