// gemm_f8.hip -- the 8-bit floating-point products with a scale for each block
// of 128: y = sum over blocks b of (x_scale[b] * w_scale[b]) * (xq wq^T)_b, for
// one matrix or for the rows of each expert, with SwiGLU on pairs of matrices.
//
// A block of K is a stage of every kernel here: its products are summed by the matrix
// units from zero (in fp32, but for mfma_codes), and the sum is scaled and added in fp32
// (4 multiply-adds for each matrix instruction, which take half of its time on the vector units).
#include <type_traits>

#include "f8_common.h"
#include "tile_device.h"
#include "tile_order.h"

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

namespace moe {

static_assert(KS == kBlock, "a stage is a block");

// 32 codes of a lane, from two 16-byte chunks of a block.
struct Codes {
  i32x4 c[2];
};
// The same in fp16, which holds every e4m3 number.
struct Wide {
  f16x8 h[4];
};
__device__ __forceinline__ Wide widen(const Codes& v) {
  Wide o;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v.c[i / 4][i % 4], 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v.c[i / 4][i % 4], 1.0f, true);
    o.h[i / 2][i % 2 * 4] = a[0];
    o.h[i / 2][i % 2 * 4 + 1] = a[1];
    o.h[i / 2][i % 2 * 4 + 2] = b[0];
    o.h[i / 2][i % 2 * 4 + 3] = b[1];
  }
  return o;
}

// The products of one block: 16 matrix rows by 16 rows of x over 128 codes of K.  Both
// operands hold the same 32 codes of K in a lane, so their order within the block does
// not matter.  In fp16 the sum is one of fp32.  The matrix units' own 8-bit products are twice
// as fast, but align the products of 8 neighbouring codes to the one with the largest exponent and
// cut off what is below 2^-13 of that (measured: 256 * 256 + 30 gives 65536 + 24); sums across those
// groups are fp32's.  Of normal values 1.2e-5 of a sum is lost, to either side alike and whatever K is: beside
// bf16's rounding, 1.6577e-3 of the outputs, the error does not change in these digits (fp16's is 2e-4).  Where large
// terms cancel it may be all of the result.  So outputs of fp32 are made from fp16, and so is everything
// that waits for memory and not for the matrix units: calls of few rows; outputs of 16 bits from tiles are
// made from codes (8192 rows of 7168 x 7168: 360 us, from fp16 in 128 x 128 tiles 830).
__device__ __forceinline__ f32x4 mfma_wide(const Wide& w, const Wide& x) {
  f32x4 c{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.h[i], x.h[i], c, 0, 0, 0);
  return c;
}
__device__ __forceinline__ f32x4 mfma_codes(const Codes& w, const Codes& x) {
  const i32x8 a = __builtin_shufflevector(w.c[0], w.c[1], 0, 1, 2, 3, 4, 5, 6, 7);
  const i32x8 b = __builtin_shufflevector(x.c[0], x.c[1], 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ void add_scaled(f32x4& acc, float s, const f32x4& v) {
#pragma unroll
  for (int c = 0; c < 4; ++c) acc[c] = fmaf(s, v[c], acc[c]);
}

// Lane (row, 16-byte column q) of a fragment in a stage of 128-byte rows: chunks q and
// 4 + q, each moved to place (chunk ^ row) & 7.
__device__ __forceinline__ Codes read_codes(const int8_t* rows, int r, int q) {
  Codes o;
#pragma unroll
  for (int h = 0; h < 2; ++h) o.c[h] = *reinterpret_cast<const i32x4*>(rows + r * KS + 16 * ((4 * h + q) ^ (r & 7)));
  return o;
}

// One wave copies a float from each lane's address to 256 bytes of LDS.
__device__ __forceinline__ void load_floats_to_lds(const float* src, float* dst) {
  __builtin_amdgcn_global_load_lds((glb_void*)src, (lds_void*)dst, 4, 0, 0);
}

// The lane's number, as something the compiler knows nothing about: what is computed from it inside a
// loop is not kept in registers throughout.
__device__ __forceinline__ int lane_here() {
  int l = threadIdx.x & 63;
  asm volatile("" : "+v"(l));
  return l;
}

// Where the scales of a matrix lie: of expert e, part p (gate, up), block `nb` of its rows.
__device__ __forceinline__ const float* w_scales(const F8Args& a, int e, int P, int p, int nb) {
  const int kb = (a.k + kBlock - 1) / kBlock, blocks = (a.n + kBlock - 1) / kBlock;
  return a.w_scale + (((size_t)e * P + p) * blocks + min(nb, blocks - 1)) * kb;
}

template <class A>
__device__ __forceinline__ void zero_rows(const A& a, const Tile& t, int i0, int cols, int threads) {
  for (int i = threadIdx.x; i < t.rows * cols; i += threads)
    if (i0 + i % cols < a.n) store_y(a.y, a.y_dtype, (size_t)y_row(a, t.p0 + i / cols) * a.n + i0 + i % cols, 0.0f);
}

// ---- few rows -------------------------------------------------------------------
//
// 16 * NN matrix rows by up to 16 rows of x a workgroup; bound by reading the matrix.  The
// NW waves take the stages in turn, each through a ring of ST buffers of its own: no
// barrier until their fp32 sums meet at the end, in the order of the waves.  The codes are
// widened to fp16: the vector units have the time.  A stage's scales come in one load: lane
// r brings that of row r of x, lane 16 + p that of part p of the matrix.
// 8 rows of N 7168, K 7168 10.8 us (4.8 TB/s), 16 of N 65536 88 us (5.4); 8 tokens with 16 of 128 experts
// each, SwiGLU of 2 x 1024, K 7168 92 us (0.63 GB: 6.8, which is what reading alone has).
template <int NN, int P, int NW, int ST>
__global__ __launch_bounds__(64 * NW, 2) void k_f8_stream(F8Args a, int tiles_n) {
  constexpr int STAGE = (1 + NN) * 16 * KS, D = 2 * (1 + NN), L = D + 1, COLS = 16 * NN / P, T = 64 * NW;
  static_assert(NN <= 2 && NW * ST * STAGE >= NW * NN * 1024, "stream");
  __shared__ __attribute__((aligned(1024))) int8_t lds[NW * ST * STAGE];
  __shared__ __attribute__((aligned(256))) float scales[NW * ST * 64];
  __shared__ int yr[16];
  Tile t;
  if (!find_tile<16>(a, blockIdx.x / tiles_n, t)) return;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i0 = blockIdx.x % tiles_n * COLS, K = a.k;
  if (t.e >= a.num_experts) {  // slots without an expert: rows of zeros
    zero_rows(a, t, i0, COLS, T);
    return;
  }
  if (threadIdx.x < 16) yr[threadIdx.x] = y_row(a, t.p0 + min((int)threadIdx.x, t.rows - 1));
  __syncthreads();
  const int lr = lane >> 3, chunk = (lane ^ lr) & 7;  // lane l of a load brings chunk (l ^ row) & 7 of row l >> 3
  const int8_t* src[D];
#pragma unroll
  for (int i = 0; i < D; ++i) {
    if (i < 2) {
      src[i] = a.x + (size_t)x_row(a, yr[8 * i + lr]) * a.x_stride;
    } else {
      const int gw = 8 * (i - 2), n = min(i0 + gw % COLS + lr, a.n - 1);  // P 2: COLS gate rows, then the up rows
      src[i] = a.w + (((size_t)t.e * P + gw / COLS) * a.n + n) * K;
    }
  }
  const bool of_x = lane < 16;
  const float* scale0 = of_x ? a.x_scale + x_row(a, yr[r]) : w_scales(a, t.e, P, min(lane - 16, P - 1), i0 / kBlock);
  const uint32_t scale_step = of_x ? (uint32_t)a.x_rows : 1u;
  const int stages = (K + KS - 1) / KS, mine = wv < stages ? (stages - wv + NW - 1) / NW : 0;
  int8_t* ring = lds + wv * ST * STAGE;
  float* sring = scales + wv * ST * 64;
  auto load = [&](int i, int b) {  // this wave's i-th stage to buffer b
    const int st = wv + NW * i, k = st * KS + 16 * chunk;
#pragma unroll
    for (int j = 0; j < D; ++j) {
      const int8_t* p = src[j] + min(k, K - 16);  // past K: zeros times codes that are there
      if (j < 2) load_to_lds(k < K ? p : kZeroCodes, ring + b * STAGE + 1024 * j);
      else load_to_lds<true>(p, ring + b * STAGE + 1024 * j);
    }
    load_floats_to_lds(scale0 + (size_t)(uint32_t)st * scale_step, sring + 64 * b);
  };
#pragma unroll
  for (int i = 0; i < ST; ++i)
    if (i < mine) load(i, i);
  f32x4 acc[NN];
#pragma unroll
  for (int j = 0; j < NN; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  int b = 0;
  Codes fw[NN], fx;
  float sx, sw[NN];
  auto read = [&]() {
    const int8_t* buf = ring + b * STAGE;
    fx = read_codes(buf, r, q);
    sx = sring[64 * b + r];
#pragma unroll
    for (int j = 0; j < NN; ++j) {
      fw[j] = read_codes(buf + 16 * KS * (1 + j), r, q);
      // P 2: with one fragment rows 0 .. 7 are the gate's and 8 .. 15 the up matrix's, with two a fragment each
      sw[j] = sring[64 * b + 16 + (P == 1 ? 0 : NN == 1 ? q / 2 : j)];
    }
    wait_lds();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&]() {
    const Wide x = widen(fx);
#pragma unroll
    for (int j = 0; j < NN; ++j) add_scaled(acc[j], sx * sw[j], mfma_wide(widen(fw[j]), x));
    b = b + 1 == ST ? 0 : b + 1;
  };
  // no branch in this loop; then what is left in the ring
  for (int st = 0; st < mine - ST; ++st) {
    wait_vm<(ST - 1) * L>();
    asm volatile("" ::: "memory");
    read();
    load(st + ST, b);
    multiply();
  }
  if (mine < ST) wait_vm<0>();
#pragma unroll
  for (int j = 0; j < ST; ++j) {
    if (j >= mine) break;
    wait_ring<ST, L>(ST - 1 - j);
    asm volatile("" ::: "memory");
    read();
    multiply();
  }
  __syncthreads();
  // register c of lane 16 q + r: matrix row 16 j + 4 q + c, row r of x
  float* red = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int j = 0; j < NN; ++j) *reinterpret_cast<f32x4*>(red + (wv * 16 + r) * (16 * NN) + 16 * j + 4 * q) = acc[j];
  __syncthreads();
  for (int i = threadIdx.x; i < t.rows * COLS; i += T) {
    const int m = i / COLS, c = i % COLS;
    if (i0 + c >= a.n) continue;
    float v[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      v[p] = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v[p] += red[(w * 16 + m) * (16 * NN) + COLS * p + c];
    }
    store_y(a.y, a.y_dtype, (size_t)yr[m] * a.n + i0 + c, P == 2 ? swiglu_f(v[0], v[P - 1]) : v[0]);
  }
}

// One float row of x, quantised on the way: each workgroup makes the row's codes and
// scales itself while the first stages of its 16 matrix rows travel, which costs less than a
// launch of its own.  Grouped: every slot reads this row.  Bound by reading the matrix and
// 2 us of start and end: N 7168, K 7168 11.1 us back to back (4.6 TB/s), N 30000 38 (5.7).
constexpr int kTokenK = 16384;  // the longest row, in whole blocks
constexpr size_t kMaxGroups = ((size_t)1 << 31) / 512;  // workgroups of a launch: its threads, and numbers in int

template <int DT, int P, int NW, int ST>
__global__ __launch_bounds__(64 * NW, 2) void k_f8_token(F8Args a, const void* __restrict__ x, int tiles_n) {
  constexpr int T = 64 * NW, STAGE = 16 * KS, L = 3, COLS = 16 / P, NC = kTokenK / 8 / T;
  __shared__ __attribute__((aligned(1024))) int8_t lds[NW * ST * STAGE];
  __shared__ __attribute__((aligned(256))) float scales[NW * ST * 64];
  __shared__ __attribute__((aligned(16))) u32x2 row[kTokenK / 8];  // the codes of x
  __shared__ float xs[kTokenK / kBlock];
  __shared__ __attribute__((aligned(16))) float red[NW][16];
  Tile t;
  if (!find_tile<16>(a, blockIdx.x / tiles_n, t)) return;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i0 = blockIdx.x % tiles_n * COLS, K = a.k;
  if (t.e >= a.num_experts) {
    zero_rows(a, t, i0, COLS, T);
    return;
  }
  // The row has arrived before the first stages are asked for, and is quantised while they travel.  (Asked for behind
  // it but not waiting for it, 7168 x 7168 took 12.3 us for 11.1, 2 x 1536, K 7168 9.8 for 7.6.)
  float v[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int at = threadIdx.x + T * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (8 * at < K) load8<DT, true>(x, at, K, v[i]);
  }
  __builtin_amdgcn_sched_barrier(0);
  const int lr = lane >> 3, chunk = (lane ^ lr) & 7;
  const int8_t* src[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int n = min(i0 + (P == 2 ? lr : 8 * i + lr), a.n - 1);  // P 2: 8 gate rows, 8 up rows
    src[i] = a.w + (((size_t)t.e * P + (P == 2 ? i : 0)) * a.n + n) * K;
  }
  const float* scale0 = w_scales(a, t.e, P, P == 2 ? q / 2 : 0, i0 / kBlock);  // the lane's own matrix rows
  const int stages = (K + KS - 1) / KS, mine = wv < stages ? (stages - wv + NW - 1) / NW : 0;
  int8_t* ring = lds + wv * ST * STAGE;
  float* sring = scales + wv * ST * 64;
  auto load = [&](int i, int b) {  // this wave's i-th stage
    const int st = wv + NW * i, k = min(st * KS + 16 * chunk, K - 16);
#pragma unroll
    for (int j = 0; j < 2; ++j) load_to_lds<true>(src[j] + k, ring + b * STAGE + 1024 * j);
    load_floats_to_lds(scale0 + st, sring + 64 * b);
  };
#pragma unroll
  for (int i = 0; i < ST; ++i)
    if (i < mine) load(i, i);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int at = threadIdx.x + T * i;
    if (at >= stages * kLanes) break;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[i][j]));
    const F8Scale s = f8_scale(block_max_bits(m));
    if (at % kLanes == 0) xs[at / kLanes] = s.stored;
    row[at] = f8_quant8(v[i], s);
  }
  wait_lds();
  meet();
  f32x4 acc{0.f, 0.f, 0.f, 0.f};
  int b = 0;
  Codes fw, fx;
  float s;
  auto read = [&](int i) {
    const int st = wv + NW * i;
#pragma unroll
    for (int h = 0; h < 2; ++h)  // the row in all 16 columns
      fx.c[h] = *reinterpret_cast<const i32x4*>(reinterpret_cast<const int8_t*>(row) + st * KS + 64 * h + 16 * q);
    fw = read_codes(ring + b * STAGE, r, q);
    const float sx = xs[st], sw = sring[64 * b + lane];
    wait_lds();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    s = sx * sw;
  };
  auto multiply = [&]() {
    add_scaled(acc, s, mfma_wide(widen(fw), widen(fx)));
    b = b + 1 == ST ? 0 : b + 1;
  };
  for (int st = 0; st < mine - ST; ++st) {
    wait_vm<(ST - 1) * L>();
    asm volatile("" ::: "memory");
    read(st);
    load(st + ST, b);
    multiply();
  }
  if (mine < ST) wait_vm<0>();
#pragma unroll
  for (int j = 0; j < ST; ++j) {
    if (j >= mine) break;
    wait_ring<ST, L>(ST - 1 - j);
    asm volatile("" ::: "memory");
    read(max(mine - ST, 0) + j);
    multiply();
  }
  if (r == 0) *reinterpret_cast<f32x4*>(&red[wv][4 * q]) = acc;
  __syncthreads();
  const int n = i0 + (int)threadIdx.x;
  if ((int)threadIdx.x >= COLS || n >= a.n) return;
  float y[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    y[p] = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) y[p] += red[w][threadIdx.x + 8 * p];
  }
  const float out = P == 2 ? swiglu_f(y[0], y[P - 1]) : y[0];
  for (int i = 0; i < t.rows; ++i) store_y(a.y, a.y_dtype, (size_t)y_row(a, t.p0 + i) * a.n + n, out);
}

bool f8_token_ok(const void* x, int k, int n, bool swiglu, int max_tiles) {
  const size_t groups = ((size_t)n * (swiglu ? 2 : 1) + 15) / 16 * max_tiles;
  return reinterpret_cast<uintptr_t>(x) % 16 == 0 && k <= kTokenK && groups < kMaxGroups;
}

template <int DT>
static void token_dt(const F8Args& a, const void* x, int max_tiles, hipStream_t s) {
  const int tiles_n = (a.n * (a.swiglu ? 2 : 1) + 15) / 16;
  const dim3 grid(tiles_n * max_tiles), block(512);
  if (a.swiglu) hipLaunchKernelGGL((k_f8_token<DT, 2, 8, 3>), grid, block, 0, s, a, x, tiles_n);
  else hipLaunchKernelGGL((k_f8_token<DT, 1, 8, 3>), grid, block, 0, s, a, x, tiles_n);
}

hipError_t launch_f8_token(const F8Args& a, const void* x, int dtype, int max_tiles, hipStream_t s) {
  if (dtype == MOE_DTYPE_BF16) token_dt<MOE_DTYPE_BF16>(a, x, max_tiles, s);
  else if (dtype == MOE_DTYPE_F16) token_dt<MOE_DTYPE_F16>(a, x, max_tiles, s);
  else token_dt<MOE_DTYPE_F32>(a, x, max_tiles, s);
  return hipGetLastError();
}

// ---- many rows: tiles through LDS ----------------------------------------------
//
// A workgroup computes BM rows of x by BN rows of the matrix (with SwiGLU BN/2
// gate rows and their BN/2 up rows, alternating by 16).  K runs in
// stages kept in ST buffers: the loads of stage k + ST - 1 are issued, straight
// into LDS, before stage k is computed.  Each wave also brings the scales of the rows of x
// that it multiplies itself, and of its matrix rows, which lie in one block.
// Bound by the matrix units under the power limit where there are tiles for all CUs: 8192 x 8192 x 7168 375 to 396 us
// on different cards (2430 to 2570 TFLOP/s; of zeros 291 to 338), by the latency of a stage where there are few: 509
// rows, SwiGLU of 2 x 1536, K 7056 28 us in 192 tiles of 64 x 128.  Products in fp16 keep the matrix units busy for 44% of
// the time instead of 68: every wave widens the codes it reads, with nearly four times the vector instructions, and adds a
// sum as soon as its products end (8192 rows of 7168 x 7168 to fp32 840 us, of zeros 770).

// One tile configuration: BM rows of x by BN matrix rows (P matrices
// interleaved), KG groups of WGM x WGN waves that take the stages in turn, ST
// buffers of a stage.  WIDE: products in fp16, for outputs of fp32; else in codes.
template <int BM_, int BN_, int WGM_, int WGN_, int KG_, int P_, int ST_, bool WIDE_>
struct TileCfg {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, KG = KG_, P = P_, ST = ST_;
  static constexpr bool WIDE = WIDE_;
  static constexpr int NW = WGM * WGN, T = 64 * NW * KG;                     // waves of a group, threads
  static constexpr int MF = BM / WGM / 16, NF = BN / WGN / 16, MO = MF / KG;  // fragments of a wave, rows of them it stores
  static constexpr bool SPLIT = BM == 64 && BN == 64;  // K may be split over workgroups
  static constexpr int STAGE = (BM + BN) * KS, RING = ST * STAGE;
  static constexpr bool TWO = RING <= 65536;             // two workgroups to a CU
  static constexpr bool ON = KG == 1 && !WIDE && !TWO;  // a workgroup goes on from tile to tile
  static constexpr int SL = MF == 4 ? 2 : 1;           // loads of a stage's scales, 64 floats each
  static constexpr int SCALES = ST * NW * SL * 64;     // floats
};

// Stores a wave's sums: its fragment rows from `first` on.  Register
// c of acc[i][j] of lane 16 q + r: matrix row 16 j + 4 q + c, row 16 i + r of x.
template <int DT, class C, class R>
__device__ __forceinline__ void tile_store(const F8Args& a, const Tile& t, const R& row_of, int i0, int wm, int wn,
                                           int first, const f32x4 (&acc)[C::MO][C::NF]) {
  constexpr int P = C::P, OB = Elem<DT>::bytes, V = 16 / OB;
  const int lane = lane_here(), r = lane & 15, q = lane >> 4;
  const bool whole = a.n % V == 0;  // 16-byte stores stay aligned, and a chunk is inside the row or outside
  const int c0 = i0 + wn * (C::BN / C::WGN / P);
#pragma unroll
  for (int i = 0; i < C::MO; ++i) {
    const int m = 16 * (C::WGM * (first + i) + wm) + r;
    if (m - r >= t.rows) break;
    const size_t row = (size_t)row_of(m) * a.n;
    // Gates below -80 are rare: the row is stored as if there were none, and once more if
    // there are.
    float lowest = 0.0f;
    auto values = [&](int j, auto low) {  // of output fragment j
      f32x4 v = acc[i][j * P];
      if constexpr (P == 2) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float u = acc[i][j * P + P - 1][c];
          lowest = fminf(lowest, v[c]);
          v[c] = decltype(low)::value ? swiglu_f(v[c], u) : swiglu_rest(v[c], u);
        }
      }
      return v;
    };
    auto put = [&](int c, const u32x4& d) {
      if (m >= t.rows) return;
      if (whole) {
        if (c < a.n) *reinterpret_cast<u32x4*>(static_cast<char*>(a.y) + (row + c) * OB) = d;
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (c + k < a.n) {
            if constexpr (OB == 4) static_cast<uint32_t*>(a.y)[row + c + k] = d[k];
            else static_cast<uint16_t*>(a.y)[row + c + k] = (uint16_t)(d[k / 2] >> (k % 2 * 16));
          }
      }
    };
    auto store = [&](auto low) {
      if constexpr (OB == 4) {
#pragma unroll
        for (int j = 0; j < C::NF / P; ++j) put(c0 + 16 * j + 4 * q, __builtin_bit_cast(u32x4, values(j, low)));
      } else {
#pragma unroll
        for (int j = 0; j < C::NF / P; j += 2) {
          if constexpr (C::NF / P > 1) {
            const f32x4 v = values(j, low), w = values(j + 1, low);
            put(c0 + 16 * j + 8 * q, join_fragments(u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])},
                                                    u32x2{pack2<DT>(w[0], w[1]), pack2<DT>(w[2], w[3])}));
          } else {  // one fragment only: 8 bytes a lane
            const f32x4 v = values(j, low);
            if (m >= t.rows) continue;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (c0 + 4 * q + k < a.n) store_y(a.y, DT, row + c0 + 4 * q + k, v[k]);
          }
        }
      }
    };
    store(std::false_type{});
    if constexpr (P == 2)
      if (__any(lowest < -80.0f)) store(std::true_type{});
  }
}

// With K split over workgroups: the sums of one part, by position, in rows of
// all tiles' columns (the matrices interleaved as in the tile).
template <class C>
__device__ __forceinline__ void tile_store_part(const F8Args& a, const Tile& t, int tn, int tiles_n, int wm, int wn,
                                                int part, int first, const f32x4 (&acc)[C::MO][C::NF]) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const size_t width = (size_t)tiles_n * C::BN;
  float* dst = a.parts + ((size_t)part * a.rows + t.p0) * width + tn * C::BN + wn * C::NF * 16 + 4 * q;
#pragma unroll
  for (int i = 0; i < C::MO; ++i) {
    const int m = 16 * (C::WGM * (first + i) + wm) + r;
    if (m >= t.rows) continue;
#pragma unroll
    for (int j = 0; j < C::NF; ++j) *reinterpret_cast<f32x4*>(dst + m * width + 16 * j) = acc[i][j];
  }
}

// The end of a tile: its outputs, or its part of the sums.
template <class C, class R>
__device__ __forceinline__ void tile_end(const F8Args& a, const Tile& t, const R& row_of, int i0, int tn, int tiles_n,
                                         int wm, int wn, int parts, int part, int first,
                                         const f32x4 (&acc)[C::MO][C::NF]) {
  if constexpr (C::SPLIT) {
    if (parts > 1) {
      tile_store_part<C>(a, t, tn, tiles_n, wm, wn, part, first, acc);
      return;
    }
  }
  if constexpr (C::WIDE) tile_store<MOE_DTYPE_F32, C>(a, t, row_of, i0, wm, wn, first, acc);
  else if (a.y_dtype == MOE_DTYPE_BF16) tile_store<MOE_DTYPE_BF16, C>(a, t, row_of, i0, wm, wn, first, acc);
  else tile_store<MOE_DTYPE_F16, C>(a, t, row_of, i0, wm, wn, first, acc);
}

template <class C>
__global__ __launch_bounds__(C::T, C::TWO ? 4 : 2) void k_f8_tile(F8Args a, int tiles_n, int tiles_m, int parts, int band_rows) {
  constexpr int BM = C::BM, BN = C::BN, WGM = C::WGM, WGN = C::WGN, P = C::P, ST = C::ST, NW = C::NW, MF = C::MF,
                KG = C::KG, NF = C::NF, GX = BM / 8, L = (BM + BN) / 8 / NW, SL = C::SL;  // L: row loads of a wave and stage
  static_assert(L * 8 * NW == BM + BN && NF % 2 == 0 && ST % KG == 0 && GX == NW * MF && (KG == 1 || NW == 4), "tile");
  constexpr bool ON = C::ON;
  // the ring, then the scales of its stages, then the rows of this tile, the next and the one before
  __shared__ __attribute__((aligned(1024))) int8_t lds[C::RING + 4 * C::SCALES + 4 * BM * (ON ? 3 : 1)];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), kg = wave / NW, wv = wave % NW;
  const int wm = wv % WGM, wn = wv / WGM, K = a.k;
  float* scales = reinterpret_cast<float*>(lds + C::RING);
  int* order = reinterpret_cast<int*>(scales + C::SCALES);
  // a grouped product's grid is sized for the most tiles its slots can make: the
  // XCDs share the ones there are
  const int count = a.order ? a.num_tiles[0] : tiles_m;
  struct Place {
    Tile t;
    int i0, tn, part;  // first output column, its tile, part of a split K
    bool any;
  };
  unsigned block = blockIdx.x;
  // The workgroup's next tile; those of slots without an expert are dealt with here.
  auto locate = [&]() {
    Place o{};
    for (;;) {
      const TileAt at = next_tile(block, gridDim.x, tiles_n, tiles_m, count, parts, band_rows);
      if (!at.any) return o;
      o.tn = at.tn;
      o.part = at.part;
      o.i0 = at.tn * (BN / P);
      if (!a.order) {
        o.t = Tile{0, at.tm * BM, min(BM, a.rows - at.tm * BM)};
      } else {
        // a scalar load, which waits for no vector load or store
        uint64_t d;
        asm volatile("s_load_dwordx2 %0, %1, 0x0\n\ts_waitcnt lgkmcnt(0)" : "=s"(d) : "s"(a.tiles + at.tm) : "memory");
        o.t.e = (int)d & 0xFFFF;
        o.t.p0 = (int)(d >> 32);
        o.t.rows = min(min((int)d >> 16, BM), a.rows - o.t.p0);
        if (o.t.e > a.num_experts || o.t.p0 < 0 || o.t.rows <= 0) continue;
        if (o.t.e == a.num_experts) {
          zero_rows(a, o.t, o.i0, BN / P, C::T);
          continue;
        }
      }
      o.any = true;
      return o;
    }
  };
  // The rows of y that a tile writes, by position in it: straight into place `at` of LDS.
  auto bring_rows = [&](const Tile& t, int at) {
    if (64 * wave < BM)
      load_floats_to_lds(reinterpret_cast<const float*>(a.order + min(t.p0 + 64 * wave + lane_here(), a.rows - 1)),
                         reinterpret_cast<float*>(order + at * BM + 64 * wave));
  };
  auto y_row_at = [&](const Tile& t, int at, int m) {
    m = min(m, t.rows - 1);
    return a.order ? (int)min((unsigned)order[at * BM + m], (unsigned)(a.rows - 1)) : t.p0 + m;
  };
  Place cur = locate();
  if (!cur.any) return;
  int place = 0;
  if (a.order) {
    bring_rows(cur.t, 0);
    wait_vm<0>();
    meet();
  }
  // Loads: a wave copies 8 rows x 128 codes at a time; lane l brings chunk
  // (l ^ row) & 7 of row l >> 3, so that the same 16-byte chunk of 8 consecutive
  // rows lies in 8 different bank groups when a fragment reads it.
  const int lr = lane >> 3, chunk = (lane ^ lr) & 7;
  // Scales: lane 16 i + r brings that of row r of the wave's fragment row i, the lanes behind
  // them (or a load of their own) those of the wave's matrix rows.
  const int8_t* src[MF];     // rows of x
  uint32_t w_off[L - MF];    // rows of the matrix, from the tile's first one: at most 255 * 65536 bytes on
  const int8_t* w_base[P];   // those first rows, the same for all lanes
  const float *scale0, *w0;
  const bool of_x = lane < 16 * MF;
  const uint32_t scale_step = of_x ? (uint32_t)a.x_rows : 1u;
  float* my_scales = scales + wv * SL * 64;
  constexpr int SW = SL == 2 ? 64 : 16 * MF;  // where the matrix's scales lie, gate and up in turn
  auto aim = [&](const Place& c, int at) {  // at a tile
    const int lane = lane_here(), lr = lane >> 3, chunk = (lane ^ lr) & 7, r = lane & 15;
#pragma unroll
    for (int i = 0; i < MF; ++i)  // a load is of 8 rows: those of x first, then the matrix's
      src[i] = a.x + (size_t)x_row(a, y_row_at(c.t, at, 8 * (wv + NW * i) + lr)) * a.x_stride + 16 * chunk;
#pragma unroll
    for (int i = 0; i < L - MF; ++i) {
      const int gw = 8 * (wv + NW * (MF + i) - GX);  // first row of the tile's matrix part; P 2: 16 gate rows, 16 up rows, ...
      const int n = min((P == 2 ? gw / 32 * 16 + gw % 16 : gw) + lr, a.n - 1 - c.i0);
      w_off[i] = (uint32_t)(n * K + 16 * chunk);
    }
#pragma unroll
    for (int p = 0; p < P; ++p) w_base[p] = a.w + (((size_t)c.t.e * P + p) * a.n + c.i0) * K;
    w0 = w_scales(a, c.t.e, P, P == 2 ? lane & 1 : 0, (c.i0 + wn * (BN / WGN / P)) / kBlock);
    scale0 = of_x ? a.x_scale + x_row(a, y_row_at(c.t, at, 16 * (WGM * (lane >> 4) + wm) + r)) : w0;
  };
  // Where this lane's chunks of the wave's first fragments and its scales lie in the buffer that is read: moved on from
  // stage to stage, so that all else are constants in the instructions and no address takes a register of its own.
  int x_at[2], w_at[2], sx_at, sw_at;
  constexpr int SCALE_STAGE = 4 * NW * SL * 64;  // bytes
  auto first_buffer = [&]() {
    const int lane = lane_here(), r = lane & 15, q = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = kg * C::STAGE + r * KS + 16 * ((4 * h + q) ^ (r & 7));
      x_at[h] = at + 16 * wm * KS;
      w_at[h] = at + (BM + wn * (BN / WGN)) * KS;
    }
    sw_at = C::RING + kg * SCALE_STAGE + 4 * wv * SL * 64;
    sx_at = sw_at + 4 * r;
  };

  // Group kg has stages kg, kg + KG, ... of the workgroup's n, its t-th in buffer KG (t % R) + kg.
  constexpr int R = ST / KG;
  const int stages = (K + KS - 1) / KS;
  const int s0 = (int)((size_t)stages * cur.part / parts), S = (int)((size_t)stages * (cur.part + 1) / parts);
  const int n = S - s0, mine = (n - kg + KG - 1) / KG, turns = (n + KG - 1) / KG;
  auto stage_of = [&](int t) { return s0 + KG * t + kg; };
  // load number i, of a row group or of scales, of stage st to buffer b; WHOLE: the stage has 128 codes
  auto load_rows = [&](int st, int b, int i, auto whole) {
    int8_t* dst = lds + b * C::STAGE + 1024 * (wv + NW * i);
    const int k = st * KS + 16 * chunk;
    constexpr bool W = decltype(whole)::value;
    if (i < MF) {  // past K: zeros on this side, times codes of the matrix that are there
      if constexpr (W) load_to_lds(src[i] + st * KS, dst);
      else load_to_lds(k >= K ? kZeroCodes : src[i] + st * KS, dst);
    } else {
      const int8_t* base = w_base[P == 2 ? (wv + NW * i - GX) / 2 % 2 : 0] + (size_t)st * KS;
      if constexpr (W) load_to_lds(base + w_off[i - MF], dst);
      else load_to_lds(base + (int)(w_off[i - MF] - (k > K - 16 ? k - (K - 16) : 0)), dst);
    }
  };
  auto load_scales = [&](int st, int b, int i) {
    float* dst = my_scales + b * (NW * SL * 64);
    if (i == 0) load_floats_to_lds(scale0 + (size_t)(uint32_t)st * scale_step, dst);
    else load_floats_to_lds(w0 + st, dst + 64);
  };
  auto first_loads = [&]() {  // of a tile: R stages
#pragma unroll
    for (int t = 0; t < R; ++t) {
      if (t >= mine) break;
#pragma unroll
      for (int i = 0; i < L; ++i) load_rows(stage_of(t), KG * t + kg, i, std::false_type{});
#pragma unroll
      for (int i = 0; i < SL; ++i) load_scales(stage_of(t), KG * t + kg, i);
    }
  };
  aim(cur, 0);
  first_loads();
  // Loads and stores complete in their order.  The first R waits of a tile are for loads that were issued
  // before the NST stores of the tile before (if it was a whole one), and leave them out: `slack` of them to come.
  constexpr int NST = ON ? C::MO * (NF / P) / 2 : 0;
  int slack = 0;
  Place next{};
  f32x4 acc[MF][NF];
  // With U of the MF fragment rows: a tile whose last rows are missing (the end of an
  // expert) neither loads nor multiplies them.
  auto run = [&](auto used) {
    constexpr int U = decltype(used)::value, LU = L - MF + U + SL;  // loads of a stage
    auto load_one = [&](int st, int b, int i, auto whole) {
      if (i >= LU - SL) load_scales(st, b, i - (LU - SL));
      else load_rows(st, b, i < U ? i : i - U + MF, whole);
    };
    auto load = [&](int st, int b) {
#pragma unroll
      for (int i = 0; i < LU; ++i) load_one(st, b, i, std::false_type{});
    };

    // The work of a stage: NF * U products in this order, column by column but for the last two
    // columns, which go row by row, so that the rows of x of the next stage can be read meanwhile.
    constexpr int F = NF * U, F0 = (NF - 2) * U;
    constexpr int LAG = C::WIDE ? 0 : F < 4 ? F - 1 : 3;
    Codes fw[4], fx[U];
    float sx[U], sw[P], scale[U][P];
    f32x4 v[LAG + 1];
    auto column = [](int f) { return f < F0 ? f / U : NF - 2 + (f - F0) % 2; };
    auto row = [](int f) { return f < F0 ? f % U : (f - F0) / 2; };
    auto read_x = [&](int i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) fx[i].c[h] = *reinterpret_cast<const i32x4*>(lds + x_at[h] + 16 * WGM * i * KS);
      sx[i] = *reinterpret_cast<const float*>(lds + sx_at + 64 * i);
    };
    auto read_w = [&](int j) {
#pragma unroll
      for (int h = 0; h < 2; ++h) fw[j % 4].c[h] = *reinterpret_cast<const i32x4*>(lds + w_at[h] + 16 * j * KS);
    };
    auto read_sw = [&]() {
#pragma unroll
      for (int p = 0; p < P; ++p) sw[p] = *reinterpret_cast<const float*>(lds + sw_at + 4 * (SW + p));
    };
    auto advance = [&](int buffers) {  // to the buffer that many further
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        x_at[h] += buffers * C::STAGE;
        w_at[h] += buffers * C::STAGE;
        asm volatile("" : "+v"(x_at[h]), "+v"(w_at[h]));
      }
      sx_at += buffers * SCALE_STAGE;
      sw_at += buffers * SCALE_STAGE;
      asm volatile("" : "+v"(sx_at), "+v"(sw_at));
    };
    // The scales that products of the stage are added with, set when the last ones of the stage before have
    // been.  With few products the next stage's are read before that: `fresh` keeps this one's.
    constexpr bool EARLY = F0 <= LAG;
    float fresh[U][P];
    auto multiply_scales = [&]() {
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int p = 0; p < P; ++p) fresh[i][p] = sx[i] * sw[p];
    };
    auto scales_of_stage = [&]() {
      if constexpr (!EARLY) multiply_scales();
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int p = 0; p < P; ++p) scale[i][p] = fresh[i][p];
    };
    auto add = [&](int f) {
      f32x4& sum = acc[row(f)][column(f)];
      add_scaled(sum, scale[row(f)][column(f) % P], v[f % (LAG + 1)]);
      asm volatile("" : "+v"(sum));  // here, and not where the compiler would gather the additions of a whole stage
    };
    // Product f, and the addition of the one LAG before it: its sum has left the matrix unit by
    // then.  (With LAG 2 a matrix instruction and its additions took 44 clocks, with 4 38, alone 35.)
    auto slot = [&](int f) {
      if constexpr (C::WIDE) {
        if (f == 0) scales_of_stage();
        add_scaled(acc[row(f)][column(f)], scale[row(f)][column(f) % P], mfma_wide(widen(fw[column(f) % 4]), widen(fx[row(f)])));
      } else {
        v[f % (LAG + 1)] = mfma_codes(fw[column(f) % 4], fx[row(f)]);
        if (f == LAG) scales_of_stage();  // those before belong to the stage before
        add(f >= LAG ? f - LAG : f - LAG + F);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    if constexpr (!C::WIDE) {
#pragma unroll
      for (int i = 0; i <= LAG; ++i) v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int p = 0; p < P; ++p) scale[i][p] = 0.0f;
    }

    // waits until all loads of this wave but those of the `later` newest stages have landed
    auto landed = [&](int later) {
      if (NST && slack > 0) {
        --slack;
        if (later >= 3) wait_vm<3 * LU + NST>();
        else if (later == 2) wait_vm<2 * LU + NST>();
        else if (later == 1) wait_vm<LU + NST>();
        else wait_vm<NST>();
      } else {
        if (later >= 3) wait_vm<3 * LU>();
        else if (later == 2) wait_vm<2 * LU>();
        else if (later == 1) wait_vm<LU>();
        else wait_vm<0>();
      }
    };
    // Of a stage's loads, FA are issued with the last columns of the stage whose buffer they take, the other FB
    // with the first columns of the next: a wave that waits to issue a load multiplies nothing.
    // (8192 x 8192 x 7168, in turn on one card: 383 us with all of them there, 375 with a third here, 368 with half; 2 x
    // 1536, K 7168, 16384 rows: 300, 296, 290.  On another card half was the slowest: 404.5, 403.4, 411; 314, 307, 310.)
    constexpr int FB = F0 > 0 ? LU / 3 : 0, FA = LU - FB;
    // The first columns; `loads`: with the rest of stage st's to buffer b.
    auto first_columns = [&](int st, int b, auto loads) {
#pragma unroll
      for (int j = 0; j < NF - 2; ++j) {
        read_w(j + 2);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int f = j * U + i;
          slot(f);
          if constexpr (decltype(loads)::value && FB > 0) {
#pragma unroll
            for (int l = 2 * f * FB / F0; l < 2 * (f + 1) * FB / F0 && l < FB; ++l) load_one(st, b, FA + l, std::true_type{});
          }
        }
      }
    };
    static_assert(NF == 2 || NF % 4 == 0, "buffers of the columns");
    // The last two columns; `next`: and the next stage's first fragments, `loads`: of stage st to buffer b.
    auto last_columns = [&](int st, int b, auto next, auto loads) {
      if constexpr (EARLY) multiply_scales();
      if constexpr (decltype(next)::value) {
        if constexpr (NF > 2) {
          read_w(0);
          read_w(1);
        }
        read_sw();
      }
#pragma unroll
      for (int g = 0; g < 2 * U; ++g) {
        slot(F0 + g);
        if constexpr (decltype(next)::value)
          if (g % 2) read_x(g / 2);
        if constexpr (decltype(loads)::value) {
#pragma unroll
          for (int i = g * FA / (2 * U); i < (g + 1) * FA / (2 * U); ++i) load_one(st, b, i, std::true_type{});
        }
      }
      if constexpr (decltype(next)::value && NF == 2) {
        read_w(0);
        read_w(1);
      }
    };
    auto first_reads = [&]() {
      read_sw();
#pragma unroll
      for (int i = 0; i < U; ++i) read_x(i);
      read_w(0);
      read_w(1);
    };
    auto pass = [&]() {  // a barrier behind which what every wave waited for has landed, and what it read is no longer needed
      wait_lds();
      meet();
    };

    first_buffer();
    landed(min(R - 1, mine - 1));
    pass();
    if (mine > 0) first_reads();
    // Stages that are followed by another and whose loads are whole ones go first.  The FB loads of the very first turn
    // bring what first_loads() has asked for already, the same bytes to the same places of stage R - 1: a copy that
    // lands while another wave reads that buffer changes nothing, since every dword it writes holds the value it
    // has, and it lands before the next stage of that buffer does, as a wave's loads do in their order.  (Leaving
    // them out by a branch spilled registers: 4096 tokens, 8 of 64 experts, SwiGLU of 2 x 1536, K 7168 1280 us for 775.)
    const int loads_whole = (K / KS - s0 - kg + KG - 1) / KG;  // of this group's stages, those of 128 codes come first
    const int ahead = min(mine, loads_whole) - (2 * R - 1);     // the pass at t loads up to stage t + 2 R - 1
    int t = 0;
    for (; t < ahead; t += R) {
#pragma unroll
      for (int u = 0; u < R; ++u) {
        first_columns(stage_of(t + u + R - 1), KG * ((u + R - 1) % R) + kg, std::true_type{});
        landed(R - 2);
        pass();
        advance(u + 1 == R ? -KG * (R - 1) : KG);
        last_columns(stage_of(t + u + R), KG * u + kg, std::true_type{}, std::true_type{});
      }
    }
    if (FB > 0 && t > 0) {
#pragma unroll
      for (int l = FA; l < LU; ++l) load_one(stage_of(t + R - 1), KG * (R - 1) + kg, l, std::true_type{});
    }
    // The rest, a stage at a time.
    for (int at = 0; t < turns; ++t, at = at + 1 == R ? 0 : at + 1) {
      const bool there = KG == 1 || t < mine;
      if (there) first_columns(0, 0, std::false_type{});
      if (t + 1 < turns) {
        landed(min(R - 2, mine - 2 - t));
        pass();
        if (t + R < mine) load(stage_of(t + R), KG * at + kg);
      } else if (ON && next.any) {  // the last stage has been read, and the next tile's rows are there
        wait_vm<0>();
        pass();
      }
      if (there) last_columns(0, 0, std::false_type{}, std::false_type{});
      if (t + 1 < mine) {
        advance(at + 1 == R ? -KG * (R - 1) : KG);
        first_reads();
      }
    }
    if constexpr (!C::WIDE) {
      if (mine > 0) {
#pragma unroll
        for (int f = F - LAG; f < F; ++f) add(f);
      }
    }
  };
  // The counts of `slack` hold for loads and stores in the order written here: none may move over these places.
  auto in_order = [&]() {
    if constexpr (!ON) return;
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  for (;;) {
    if constexpr (ON) {
      next = locate();
      if (next.any && a.order) bring_rows(next.t, place == 2 ? 0 : place + 1);
    }
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int need = (cur.t.rows + 16 * WGM - 1) / (16 * WGM);
    if (need >= MF) run(std::integral_constant<int, MF>{});
    else if (MF == 4 && need == 3) run(std::integral_constant<int, MF == 4 ? 3 : 1>{});
    else if (MF == 4 && need == 2) run(std::integral_constant<int, MF == 4 ? 2 : 1>{});
    else run(std::integral_constant<int, 1>{});
    if constexpr (ON) {
      if (next.any) {  // its first stages travel while this tile's outputs are stored
        aim(next, place == 2 ? 0 : place + 1);
        first_loads();
      }
    }
    in_order();
    auto row_of = [&](int m) { return y_row_at(cur.t, place, m); };
    if constexpr (KG == 1) {
      tile_end<C>(a, cur.t, row_of, cur.i0, cur.tn, tiles_n, wm, wn, parts, cur.part, 0, acc);
      in_order();
    } else {
      // each group gives the other half of its fragment rows away and adds what it gets
      f32x4* swap = reinterpret_cast<f32x4*>(lds) + (wv * C::MO * NF) * 64 + lane;
      constexpr int HALF = NW * C::MO * NF * 64;
      static_assert(2 * HALF * 16 <= C::RING, "sums");
      f32x4 sum[C::MO][NF];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < C::MO; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const f32x4 lower = acc[i][j], upper = acc[C::MO + i][j];  // values: a choice between places would keep acc in memory
          f32x4 away;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            sum[i][j][c] = kg ? upper[c] : lower[c];
            away[c] = kg ? lower[c] : upper[c];
          }
          swap[kg * HALF + (i * NF + j) * 64] = away;
        }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < C::MO; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) sum[i][j] += swap[(1 - kg) * HALF + (i * NF + j) * 64];
      tile_end<C>(a, cur.t, row_of, cur.i0, cur.tn, tiles_n, wm, wn, parts, cur.part, kg * C::MO, sum);
    }
    if (!ON || !next.any) break;
    const bool all_stores = cur.t.rows == BM && cur.i0 + BN / P <= a.n && a.n % 8 == 0;
    slack = all_stores ? R : 0;
    cur = next;
    place = place == 2 ? 0 : place + 1;
  }
}

constexpr int kMaxParts = 8;

// The parts of a split K (of a dense product) added up in their order and stored: a
// workgroup takes 4 rows, a wave each, by 256 columns.
template <int P>
__global__ __launch_bounds__(256) void k_f8_parts(F8Args a, int parts, int tiles_n, int cols) {
  constexpr int BN = 64, BO = BN / P;
  const int m = blockIdx.x / cols * 4 + (threadIdx.x >> 6), n = blockIdx.x % cols * 256 + (threadIdx.x & 63) * 4;
  if (m >= a.rows || n >= a.n) return;
  const size_t width = (size_t)tiles_n * BN, step = (size_t)a.rows * width;
  const float* src = a.parts + (size_t)m * width + n / BO * BN + n % BO / 16 * 16 * P + n % 16;
  f32x4 v[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    f32x4 sum{0.f, 0.f, 0.f, 0.f}, part[kMaxParts];  // all parts requested before the first is added
#pragma unroll
    for (int i = 0; i < kMaxParts; ++i)
      part[i] = *reinterpret_cast<const f32x4*>(src + min(i, parts - 1) * step + 16 * p);
#pragma unroll
    for (int i = 0; i < kMaxParts; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) sum[c] += i < parts ? part[i][c] : 0.0f;
    v[p] = sum;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (n + k < a.n) store_y(a.y, a.y_dtype, (size_t)m * a.n + n + k, P == 2 ? swiglu_f(v[0][k], v[P - 1][k]) : v[0][k]);
}

template <class C>
static void tile_launch(const F8Args& a, int max_tiles, int parts, hipStream_t s) {
  const int tiles_n = (a.n * C::P + C::BN - 1) / C::BN;
  const int per_xcd = (tiles_n * max_tiles * parts + 7) / 8;
  int band = 8;
  if (a.order) {
    band = (a.rows / a.num_experts + C::BM / 2) / C::BM;
    band = band < 1 ? 1 : band > 8 ? 8 : band;
  }
  int grid = 8 * per_xcd;
  if (C::ON) {
    const int resident = (num_cus() + 7) / 8 * 8;
    grid = grid < resident ? grid : resident;
  }
  hipLaunchKernelGGL(k_f8_tile<C>, dim3(grid), dim3(C::T), 0, s, a, tiles_n, max_tiles, parts, band);
  if constexpr (C::SPLIT) {
    if (parts == 1) return;
    const int cols = (a.n + 255) / 256;
    hipLaunchKernelGGL(k_f8_parts<C::P>, dim3(cols * ((a.rows + 3) / 4)), dim3(256), 0, s, a, parts, tiles_n, cols);
  }
}

// 32 matrix rows a workgroup, or 16 where all those have a CU to themselves (8 rows of K 7168: N 1536, 96
// of them, 6.8 us for 8.9, SwiGLU of 2 x 1536, 192, 8.6 for 9.4; N 7168, 448, 12.5 for 10.8; 37 rows of N 1536, 288,
// 10.1 for 8.8).
template <int NN, int NW, int ST>
static void stream_launch_as(const F8Args& a, int max_tiles, hipStream_t s) {
  const int tiles_n = (a.n * (a.swiglu ? 2 : 1) + 16 * NN - 1) / (16 * NN);
  const dim3 grid(tiles_n * max_tiles), block(64 * NW);
  if (a.swiglu) hipLaunchKernelGGL((k_f8_stream<NN, 2, NW, ST>), grid, block, 0, s, a, tiles_n);
  else hipLaunchKernelGGL((k_f8_stream<NN, 1, NW, ST>), grid, block, 0, s, a, tiles_n);
}

static void stream_launch(const F8Args& a, int max_tiles, hipStream_t s) {
  const int rows = a.n * (a.swiglu ? 2 : 1), halves = (rows + 15) / 16;
  if (halves * max_tiles <= 256) stream_launch_as<1, 4, 3>(a, max_tiles, s);
  else stream_launch_as<2, 4, 2>(a, max_tiles, s);
}

// The kernels a product may run on, in the order of F8Plan::kind: 16 rows of x by 32
// matrix rows as a stream, and the tiles.
struct Tiling {
  int bm, bn;
  int resident;            // workgroups that the card holds at a time
  bool rounds;             // dense: time goes by whole rounds of them
  double d0, d1;           // dense: us a round, and a stage of a round
  double g0, g1, g2, g3, g4;  // grouped, see f8_plan
};
// With the products of codes, and with those in fp16 (the last two tiles: not for these).
constexpr Tiling kTilings[2][6] = {{{16, 32, 512, false, 3.5, 0.157, 1.2, 1.25, 0.226, 0.0, 0.075},
                                    {64, 64, 256, true, 3.55, 0.205, 0.5, 2.9, 0.109, 0.146, 0.422},
                                    {64, 128, 256, true, 3.7, 0.3, 0.0, 3.55, 0.173, 0.103, 0.374},
                                    {128, 128, 256, true, 4.2, 0.49, 0.0, 5.43, 0.118, 0.379, 0.389},
                                    {128, 128, 512, false, 4.5, 1.15, 0.0, 3.59, 0.665, 0.0, 0.418},
                                    {256, 256, 256, true, 7.0, 1.17, 0.0, 8.42, 0.784, 0.0, 0.314}},
                                   {{16, 32, 512, false, 3.3, 0.084, 3.46, 0.457, 0.246, 0.0, 0.067},
                                    {64, 64, 256, true, 3.55, 0.21, 0.4, 3.69, 0.118, 0.164, 0.458},
                                    {64, 128, 256, true, 4.0, 0.3, 0.0, 3.97, 0.153, 0.182, 0.905},
                                    {128, 128, 256, true, 3.73, 0.456, 0.0, 4.33, 0.118, 0.535, 0.646}}};
constexpr int kStream = 0, kSplit = 1, kTwoToACu = 4, kKinds[2] = {6, 4};

// Which kernel a product runs on: the one with the least estimated time.
// Dense: T workgroups in rounds of those that the card holds, each d0 + d1 * stages.  Up
// to 16 rows always the stream; with more rows it reads the matrix again for every 16, and is
// taken where the card holds all its workgroups.  Two 128 x 128 tiles to a CU (two
// buffers of a stage each) are for more than one round of single ones (four buffers).
// Measured at N 7168, K 7168: 8 rows 10.6 us (64 x 64 tiles 15.3), 24 rows 19.6; 128 rows:
// 64 x 64 21.1 us, 64 x 128 28.2, 128 x 128 37.5; 2048 rows: 234, 172, 136 (two to a CU 124),
// 256 x 256 94; 8192 rows: 864, 642, 489, 451, 366.
// Grouped: each expert's matrix comes from HBM, an expert's rows end anywhere in a tile
// (half a tile more on average, of which only the rows that there are cost anything).
// g0 + rounds * (g1 + g2 * stages) + g3 * stages * rounds' worth of rows + g4 * the time to read
// the matrices at 6.6 TB/s.  106 experts of 9 rows, 2 x 4172, K 256: the stream 99 us, 64 x 64 93,
// 128 x 128 40 (two to a CU 35), 256 x 256 41; 12 rows of 84 experts, N 92, K 6112: 6.6, 11.9, 20, 22, 32.
// Fitted to 1153 products of the sizes in 1 to 8192 rows, N 64 to 8192, K 64 to 8192, 2 to 128
// experts; on 500 others the choice costs 1.6% over the best kernel on average where it is dense
// (2.1% in fp16), 5.0% (3.9%) where it is grouped.
// K is split over parts where 64 x 64 tiles leave most CUs without work and the stages saved
// are worth adding the parts up (64 rows of N 7168, K 7168: 18.3 us in 2 parts, 21.1 in one;
// 37 rows of N 1536, K 7168 to fp32: 10.9 in 8 parts, 20.7 in one, 8.9 as a stream).
F8Plan f8_plan(int rows, int experts, bool grouped, int n, int k, bool swiglu, bool wide) {
  const int P = swiglu ? 2 : 1, stages = (k + KS - 1) / KS, used = !grouped ? 1 : rows < experts ? rows : experts;
  const double per = (double)rows / used, read = (double)used * n * P * k / 6.6e6;
  F8Plan best{-1, 0, 1, 0};
  double least = 0.0;
  bool launchable = false;
  for (int kind = 0; kind < kKinds[wide]; ++kind) {
    const Tiling& m = kTilings[wide][kind];
    const int cols = (n * P + m.bn - 1) / m.bn;
    double time;
    int parts = 1;
    if (grouped) {
      const double down = per / m.bm + 0.5 < 1.0 ? 1.0 : per / m.bm + 0.5;
      double load = down * used * cols / m.resident, work = (per / m.bm + 0.25) * used * cols / m.resident;
      if (kind > kSplit) load = ceil(load);
      if (load < 1.0) load = 1.0;
      if (work < 1.0) work = 1.0;
      time = m.g0 + (m.g1 + m.g2 * stages) * load + m.g3 * stages * work + m.g4 * read;
      if (kind != kStream && time < 1.2 * read) time = 1.2 * read;
    } else {
      const double tiles = (double)((rows + m.bm - 1) / m.bm) * cols;
      if (kind == kStream ? rows > 16 && tiles > m.resident : kind == kTwoToACu && tiles <= 256.0) continue;
      double load = m.rounds ? ceil(tiles / m.resident) : tiles / m.resident;
      if (load < 1.0) load = 1.0;
      time = kind == kStream && rows <= 16 ? 0.0 : (m.d0 + m.d1 * stages) * load;
      if (kind == kSplit) {
        parts = (int)(224.0 / tiles);
        if (parts > kMaxParts) parts = kMaxParts;
        if (parts > stages / 6) parts = stages / 6;
        const double saved = parts > 1 ? m.d1 * (stages - stages / parts) - 4.0 : 0.0;
        if (saved <= 0.0) parts = 1;
        else time -= saved;
      }
    }
    // a kernel whose workgroups a launch does not hold only where no other one's fit either
    const bool fits = (size_t)cols * parts * (grouped ? max_tiles(rows, experts, m.bm) : (rows + m.bm - 1) / m.bm) < kMaxGroups;
    if (best.kind >= 0 && (fits == launchable ? time >= least : launchable)) continue;
    least = time;
    launchable = fits;
    best = F8Plan{kind, m.bm, parts, parts > 1 ? (size_t)parts * rows * cols * m.bn * 4 : 0};
  }
  return best;
}

template <int P, bool WIDE>
static void tiles_launch(const F8Args& a, const F8Plan& plan, int max_tiles, hipStream_t s) {
  if (plan.kind == 1) tile_launch<TileCfg<64, 64, 2, 2, 2, P, 8, WIDE>>(a, max_tiles, plan.parts, s);
  else if (plan.kind == 2) tile_launch<TileCfg<64, 128, 2, 2, 2, P, 6, WIDE>>(a, max_tiles, 1, s);
  else if (plan.kind == 3) tile_launch<TileCfg<128, 128, 4, 2, 1, P, 4, WIDE>>(a, max_tiles, 1, s);
  else if constexpr (!WIDE) {
    if (plan.kind == kTwoToACu) tile_launch<TileCfg<128, 128, 4, 2, 1, P, 2, WIDE>>(a, max_tiles, 1, s);
    else tile_launch<TileCfg<256, 256, 4, 2, 1, P, 2, WIDE>>(a, max_tiles, 1, s);
  }
}

bool f8_launchable(const F8Plan& plan, int n, bool swiglu, int max_tiles) {
  const size_t bn = kTilings[0][plan.kind].bn, cols = ((size_t)n * (swiglu ? 2 : 1) + bn - 1) / bn;
  return cols * max_tiles * plan.parts < kMaxGroups;
}

hipError_t launch_gemm_f8(const F8Args& a, const F8Plan& plan, int max_tiles, hipStream_t s) {
  const bool wide = a.y_dtype == MOE_DTYPE_F32;
  if (plan.kind == kStream) stream_launch(a, max_tiles, s);
  else if (a.swiglu) wide ? tiles_launch<2, true>(a, plan, max_tiles, s) : tiles_launch<2, false>(a, plan, max_tiles, s);
  else wide ? tiles_launch<1, true>(a, plan, max_tiles, s) : tiles_launch<1, false>(a, plan, max_tiles, s);
  return hipGetLastError();
}

}  // namespace moe
