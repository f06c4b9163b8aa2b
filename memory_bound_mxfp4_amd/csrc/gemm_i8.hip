// gemm_i8.hip -- the 8-bit integer products: y = x_scale * w_scale * (xq wq^T),
// for one matrix or for the rows of each expert, with SwiGLU on pairs of
// matrices.  Sums are int32 and exact, so neither the split of K nor its
// order changes a result.
#include "i8_common.h"

namespace moe {

// The row that position p of a product reads and the one it writes.  Dense:
// both p.  Grouped: position p of the order names a slot, which is the row
// written; the row read is the slot (FC2) or its token (FC1)
// (clamped: whatever a groups buffer holds, no address leaves x or y).
__device__ __forceinline__ int y_row(const I8Args& a, int p) {
  return a.order ? (int)min((unsigned)a.order[p], (unsigned)(a.rows - 1)) : p;
}
__device__ __forceinline__ int x_row(const I8Args& a, int yr) { return a.x_div > 1 ? yr / a.x_div : yr; }

// The tile of rows a workgroup works on: expert, first position, positions.
struct Tile {
  int e, p0, rows;
};

template <int BM>
__device__ __forceinline__ bool find_tile(const I8Args& a, int t, Tile& o) {
  if (!a.order) {
    o.e = 0;
    o.p0 = t * BM;
    o.rows = min(BM, a.rows - o.p0);
    return true;
  }
  if (t >= a.num_tiles[0]) return false;
  o.e = a.tiles[t].x;
  o.p0 = a.tiles[t].y;
  if ((unsigned)o.e > (unsigned)a.num_experts || (unsigned)o.p0 >= (unsigned)a.rows) return false;
  o.rows = min(min(BM, a.offsets[o.e + 1] - o.p0), a.rows - o.p0);
  return o.rows > 0;
}

// 16 weight rows (of each of P matrices) by up to 16 * NCG rows of x.  Both
// operands come straight from memory as the matrix instruction takes them:
// lane 16 q + r holds 16 codes of weight row r and of activation row r.  The
// four waves split K into 256-byte segments; their int32 sums meet in LDS.
template <int NCG, int P>
__global__ __launch_bounds__(256) void k_i8_direct(I8Args a) {
  __shared__ int red[4][P][NCG][16][16];
  Tile t;
  if (!find_tile<16 * NCG>(a, blockIdx.y, t)) return;
  const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16, K = a.k;
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
  if (t.e >= a.num_experts) {  // slots without an expert: rows of zeros
#pragma unroll
    for (int c = 0; c < NCG; ++c)
      if (16 * c + row < t.rows && n0 + col < a.n)
        store_y(a.y, a.y_dtype, (size_t)y_row(a, t.p0 + 16 * c + row) * a.n + n0 + col, 0.0f);
    return;
  }
  const int8_t* wp[P];
#pragma unroll
  for (int p = 0; p < P; ++p) wp[p] = a.w + (((size_t)t.e * P + p) * a.n + min(n0 + r, a.n - 1)) * K;
  const int8_t* xp[NCG];
#pragma unroll
  for (int c = 0; c < NCG; ++c)
    xp[c] = a.x + (size_t)x_row(a, y_row(a, t.p0 + min(16 * c + r, t.rows - 1))) * a.x_stride;
  i32x4 acc[P][NCG];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int c = 0; c < NCG; ++c) acc[p][c] = i32x4{0, 0, 0, 0};
  const i32x4 z{0, 0, 0, 0};
  for (int s = wv * 256; s < K; s += 1024) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = s + 64 * j + 16 * q, kc = min(k, K - 16);
      i32x4 xv[NCG];
#pragma unroll
      for (int c = 0; c < NCG; ++c) xv[c] = *reinterpret_cast<const i32x4*>(xp[c] + kc);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        i32x4 wvv = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(wp[p] + kc));
        if (k >= K) wvv = z;
#pragma unroll
        for (int c = 0; c < NCG; ++c) acc[p][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wvv, xv[c], acc[p][c], 0, 0, 0);
      }
    }
  }
  // accumulator register i of lane 16 q + r: weight row 4 q + i, activation row r
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int c = 0; c < NCG; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wv][p][c][r][4 * q + i] = acc[p][c][i];
  __syncthreads();
#pragma unroll
  for (int c = 0; c < NCG; ++c) {
    if (16 * c + row >= t.rows || n0 + col >= a.n) continue;
    const int yr = y_row(a, t.p0 + 16 * c + row);
    const float sx = a.x_scale[x_row(a, yr)];
    float v[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int sum = red[0][p][c][row][col] + red[1][p][c][row][col] + red[2][p][c][row][col] + red[3][p][c][row][col];
      v[p] = (float)sum * (sx * a.w_scale[((size_t)t.e * P + p) * a.n + n0 + col]);
    }
    store_y(a.y, a.y_dtype, (size_t)yr * a.n + n0 + col, P == 2 ? swiglu_f(v[0], v[P - 1]) : v[0]);
  }
}

int i8_tile_rows(const I8Args& a) { return a.rows <= 16 ? 16 : 64; }

hipError_t launch_gemm_i8(const I8Args& a, int tile_rows, int max_tiles, hipStream_t s) {
  const dim3 grid((a.n + 15) / 16, max_tiles), block(256);
  if (tile_rows == 16) {
    if (a.swiglu) hipLaunchKernelGGL((k_i8_direct<1, 2>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_i8_direct<1, 1>), grid, block, 0, s, a);
  } else {
    if (a.swiglu) hipLaunchKernelGGL((k_i8_direct<4, 2>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_i8_direct<4, 1>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace moe
