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

// ---- many rows: tiles through LDS ----------------------------------------------
//
// A workgroup computes BM rows of x by BN rows of the matrix (with SwiGLU BN/2
// gate rows and their BN/2 up rows, alternating by 16).  K runs in stages of
// 64 codes, kept in ST buffers: the loads of stage k + ST - 1 are issued, straight into
// LDS, before stage k is computed.
constexpr int KS = 64;

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void glb_void;

// 16 codes of zero: what a lane reads in place of codes of x past K.
__device__ const __attribute__((aligned(16))) int8_t kZeroCodes[16] = {0};

// One wave copies 64 x 16 bytes from its lanes' addresses to 1 KB of LDS.
__device__ __forceinline__ void load_to_lds(const int8_t* src, int8_t* dst) {
  __builtin_amdgcn_global_load_lds((glb_void*)src, (lds_void*)dst, 16, 0, 0);
}

// Waits until at most VM of the wave's loads are out, and for its LDS reads.
template <int VM>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4));
}

template <int DT>
__device__ __forceinline__ void store4(void* y, size_t i, const float* v) {
  if constexpr (DT == MOE_DTYPE_F32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(y) + i) = f32x4{v[0], v[1], v[2], v[3]};
  } else {
    uint32_t h[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) h[c] = DT == MOE_DTYPE_BF16 ? f32_to_bf16(v[c]) : f32_to_f16(v[c]);
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(y) + i) = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
  }
}

// Scales a wave's sums and stores them.  Register c of acc[i][j] of lane
// 16 q + r: matrix row 16 j + 4 q + c, row 16 i + r of x.
template <int DT, int BM, int BN, int WGM, int WGN, int P>
__device__ __forceinline__ void tile_store(const I8Args& a, const Tile& t, int i0, int wm, int wn,
                                           const i32x4 (&acc)[BM / WGM / 16][BN / WGN / 16]) {
  constexpr int MF = BM / WGM / 16, NF = BN / WGN / 16;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const bool vec = a.n % 4 == 0;
  const float* sw = a.w_scale + (size_t)t.e * P * a.n;
#pragma unroll
  for (int j = 0; j < NF; j += P) {
    const int n = i0 + (wn * (BN / WGN) + 16 * j) / P + 4 * q;
    float s[P][4];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[p][c] = sw[p * a.n + min(n + c, a.n - 1)];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = wm * (BM / WGM) + 16 * i + r;
      if (m >= t.rows) continue;
      const int yr = y_row(a, t.p0 + m);
      const float sx = a.x_scale[x_row(a, yr)];
      const size_t at = (size_t)yr * a.n + n;
      float v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[c] = (float)acc[i][j][c] * (sx * s[0][c]);
        if (P == 2) v[c] = swiglu_f(v[c], (float)acc[i][j + P - 1][c] * (sx * s[P - 1][c]));
      }
      if (vec) {
        if (n < a.n) store4<DT>(a.y, at, v);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (n + c < a.n) store_y(a.y, DT, at + c, v[c]);
      }
    }
  }
}

template <int BM, int BN, int WGM, int WGN, int P, int ST>
__global__ __launch_bounds__(64 * WGM * WGN) void k_i8_tile(I8Args a, int tiles_n, int m_tiles) {
  constexpr int NW = WGM * WGN, MF = BM / WGM / 16, NF = BN / WGN / 16;  // fragments of a wave
  constexpr int LX = BM / 16 / NW, LW = BN / 16 / NW, L = LX + LW;       // loads of a wave and stage
  static_assert(LX * 16 * NW == BM && LW * 16 * NW == BN && NF % P == 0, "tile");
  __shared__ __attribute__((aligned(1024))) int8_t lds[ST][(BM + BN) * KS];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wv % WGM, wn = wv / WGM;
  const int tn = blockIdx.x % tiles_n, tm = blockIdx.x / tiles_n;
  Tile t;
  if (!find_tile<BM>(a, tm, t)) return;
  const int K = a.k, i0 = tn * (BN / P);  // first output column
  if (t.e >= a.num_experts) {
    for (int m = threadIdx.x / 64; m < t.rows; m += NW)
      for (int n = i0 + lane; n < min(i0 + BN / P, a.n); n += 64)
        store_y(a.y, a.y_dtype, (size_t)y_row(a, t.p0 + m) * a.n + n, 0.0f);
    return;
  }
  // Loads: a wave copies 16 rows x 64 codes at a time; lane l brings chunk
  // (l & 3) ^ swz of row l >> 2, so that the 16-byte chunks of consecutive rows
  // lie in different banks when a fragment reads one chunk of 16 rows.
  const int lr = lane >> 2, chunk = (lane & 3) ^ ((lr >> 1) & 3);
  const int8_t* src[L];
#pragma unroll
  for (int i = 0; i < LX; ++i) {
    const int m = min(16 * (wv + NW * i) + lr, t.rows - 1);
    src[i] = a.x + (size_t)x_row(a, y_row(a, t.p0 + m)) * a.x_stride;
  }
#pragma unroll
  for (int i = 0; i < LW; ++i) {
    const int g = wv + NW * i;  // group of 16 tile rows
    const int n = min(i0 + (P == 2 ? 16 * (g >> 1) : 16 * g) + lr, a.n - 1);
    src[LX + i] = a.w + (((size_t)t.e * P + (P == 2 ? g & 1 : 0)) * a.n + n) * K;
  }
  const int S = (K + KS - 1) / KS;
  auto load = [&](int st) {
    int8_t* buf = lds[st % ST];
    const int k = st * KS + 16 * chunk;
    if ((st + 1) * KS <= K) {
#pragma unroll
      for (int i = 0; i < L; ++i)
        load_to_lds(src[i] + k, buf + (i < LX ? 1024 * (wv + NW * i) : BM * KS + 1024 * (wv + NW * (i - LX))));
    } else {  // the last stage of a K that is no multiple of 64: zeros past K on x's side
#pragma unroll
      for (int i = 0; i < L; ++i)
        load_to_lds(i < LX && k >= K ? kZeroCodes : src[i] + min(k, K - 16),
                    buf + (i < LX ? 1024 * (wv + NW * i) : BM * KS + 1024 * (wv + NW * (i - LX))));
    }
  };
  i32x4 acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
#pragma unroll
  for (int st = 0; st < ST - 1; ++st)
    if (st < S) load(st);
  const int frag = r * KS + 16 * (q ^ ((r >> 1) & 3));
  for (int st = 0; st < S; ++st) {
    // stage st has landed when at most the loads of the stages after it are out
    const int later = min(ST - 2, S - 1 - st);
    if (later == 2) wait_vm<2 * L>();
    else if (later == 1) wait_vm<L>();
    else wait_vm<0>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // every wave is past stage st - 1: its buffer takes stage st + ST - 1
    if (st + ST - 1 < S) load(st + ST - 1);
    const int8_t* bx = lds[st % ST] + wm * (BM / WGM) * KS + frag;
    const int8_t* bw = lds[st % ST] + BM * KS + wn * (BN / WGN) * KS + frag;
    i32x4 fw[NF], fx[MF];
#pragma unroll
    for (int j = 0; j < NF; ++j) fw[j] = *reinterpret_cast<const i32x4*>(bw + 1024 * j);
#pragma unroll
    for (int i = 0; i < MF; ++i) fx[i] = *reinterpret_cast<const i32x4*>(bx + 1024 * i);
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[j], fx[i], acc[i][j], 0, 0, 0);
  }
  if (a.y_dtype == MOE_DTYPE_BF16) tile_store<MOE_DTYPE_BF16, BM, BN, WGM, WGN, P>(a, t, i0, wm, wn, acc);
  else if (a.y_dtype == MOE_DTYPE_F16) tile_store<MOE_DTYPE_F16, BM, BN, WGM, WGN, P>(a, t, i0, wm, wn, acc);
  else tile_store<MOE_DTYPE_F32, BM, BN, WGM, WGN, P>(a, t, i0, wm, wn, acc);
}

int i8_tile_rows(const I8Args& a) {
  if (a.rows <= 16) return 16;
  const int per = a.order ? a.rows / a.num_experts : a.rows;
  return per >= 128 ? 256 : per > 16 ? 64 : 16;
}

template <int BM, int BN, int WGM, int WGN, int P, int ST>
static void tile_launch(const I8Args& a, int max_tiles, hipStream_t s) {
  const int tiles_n = (a.n * P + BN - 1) / BN;
  hipLaunchKernelGGL((k_i8_tile<BM, BN, WGM, WGN, P, ST>), dim3(tiles_n * max_tiles), dim3(64 * WGM * WGN), 0, s, a,
                     tiles_n, max_tiles);
}

hipError_t launch_gemm_i8(const I8Args& a, int tile_rows, int max_tiles, hipStream_t s) {
  if (tile_rows == 256) {
    if (a.swiglu) tile_launch<256, 256, 2, 4, 2, 4>(a, max_tiles, s);
    else tile_launch<256, 256, 2, 4, 1, 4>(a, max_tiles, s);
    return hipGetLastError();
  }
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
