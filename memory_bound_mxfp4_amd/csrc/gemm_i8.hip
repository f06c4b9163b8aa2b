// gemm_i8.hip -- the 8-bit integer products: y = x_scale * w_scale * (xq wq^T),
// for one matrix or for the rows of each expert, with SwiGLU on pairs of
// matrices.  Sums are int32 and exact, so neither the split of K nor its
// order changes a result.
#include <type_traits>

#include "i8_common.h"
#include "tile_order.h"

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
  // both loads at once: an entry past the number of tiles is inside the buffer
  const int n = a.num_tiles[0];
  const int2 d = a.tiles[t];
  o.e = d.x & 0xFFFF;
  o.p0 = d.y;
  o.rows = min(min(d.x >> 16, BM), a.rows - o.p0);
  return t < n && o.e <= a.num_experts && o.p0 >= 0 && o.rows > 0;
}

// Codes of K that a wave or workgroup moves at a time: a whole cache line of
// every row.  (With 64 codes, each line crosses from L2 twice: the few-rows
// kernel reached 4.3 TB/s that way, see below.)
constexpr int KS = 128;

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void glb_void;

// 16 codes of zero: what a lane reads in place of codes of x past K.
__device__ const __attribute__((aligned(16))) int8_t kZeroCodes[16] = {0};

// One wave copies 64 x 16 bytes from its lanes' addresses to 1 KB of LDS.
// NT: not kept in the caches (a matrix that is read once).
template <bool NT = false>
__device__ __forceinline__ void load_to_lds(const int8_t* src, int8_t* dst) {
  __builtin_amdgcn_global_load_lds((glb_void*)src, (lds_void*)dst, 16, 0, NT ? 2 : 0);
}

// Waits until at most VM of the wave's loads are out, and for its LDS reads.
template <int VM>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4));
}

// Waits until at most the newest n of a ring's stages are out; n is a constant
// where this is called.
template <int ST, int L>
__device__ __forceinline__ void wait_ring(int n) {
  static_assert(ST <= 4, "ring");
  if (n >= 3) wait_vm<3 * L>();
  else if (n == 2) wait_vm<2 * L>();
  else if (n == 1) wait_vm<L>();
  else wait_vm<0>();
}

// Waits for the wave's LDS reads alone.
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }

// Barrier of the workgroup that neither memory accesses nor multiplications cross.
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// ---- few rows -------------------------------------------------------------------
//
// 16 * NN matrix rows by up to 16 rows of x a workgroup; bound by reading
// the matrix.  The NW waves take stages of K in turn, each through a ring of ST
// buffers of its own: no barrier until their int32 sums meet at the end, and a
// buffer is loaded again as soon as its fragments are in registers.
// N 7168, K 7168, 8 rows: 10.2 us (5 TB/s, 2.5 us of it start and end); N 65536: 72 us
// (6.5 TB/s); 8 tokens with 16 of 128 experts each, 2 x 1024, K 7168: 91 to 97 us (6.4 TB/s).
// (Waves that share a buffer and meet at every stage reached 5.2 TB/s.  Two buffers a
// wave, three workgroups to a CU, are as fast as three for long K and better for
// short: 128 experts, N 7168, K 1024, 72 us for 86.)
template <int NN, int P, int NW, int ST>
__global__ __launch_bounds__(64 * NW) void k_i8_stream(I8Args a, int tiles_n) {
  constexpr int STAGE = (1 + NN) * 16 * KS, L = 2 * (1 + NN), COLS = 16 * NN / P, T = 64 * NW;
  static_assert(NN <= 2 && NW * ST * STAGE >= NW * NN * 1024, "stream");
  __shared__ __attribute__((aligned(1024))) int8_t lds[NW * ST * STAGE];
  __shared__ float scales[16 * (NN + 1)];
  __shared__ int yr[16];
  Tile t;
  if (!find_tile<16>(a, blockIdx.x / tiles_n, t)) return;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i0 = blockIdx.x % tiles_n * COLS, K = a.k;
  if (t.e >= a.num_experts) {  // slots without an expert: rows of zeros
    for (int i = threadIdx.x; i < t.rows * COLS; i += T)
      if (i0 + i % COLS < a.n) store_y(a.y, a.y_dtype, (size_t)y_row(a, t.p0 + i / COLS) * a.n + i0 + i % COLS, 0.0f);
    return;
  }
  if (threadIdx.x < 16) yr[threadIdx.x] = y_row(a, t.p0 + min((int)threadIdx.x, t.rows - 1));
  __syncthreads();
  // lane l of a load brings chunk (l ^ row) & 7 of row l >> 3, as in the tiles below
  const int lr = lane >> 3, chunk = (lane ^ lr) & 7;
  const int8_t* src[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    if (i < 2) {
      src[i] = a.x + (size_t)x_row(a, yr[8 * i + lr]) * a.x_stride;
    } else {
      const int gw = 8 * (i - 2), n = min(i0 + gw % COLS + lr, a.n - 1);  // P 2: COLS gate rows, then the up rows
      src[i] = a.w + (((size_t)t.e * P + gw / COLS) * a.n + n) * K;
    }
  }
  const int stages = (K + KS - 1) / KS, mine = wv < stages ? (stages - wv + NW - 1) / NW : 0;
  int8_t* ring = lds + wv * ST * STAGE;
  auto load = [&](int i, int8_t* buf) {  // this wave's i-th stage
    const int k = (wv + NW * i) * KS + 16 * chunk;
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const int8_t* p = src[j] + min(k, K - 16);
      if (j < 2) load_to_lds(k < K ? p : kZeroCodes, buf + 1024 * j);
      else load_to_lds<true>(p, buf + 1024 * j);
    }
  };
#pragma unroll
  for (int i = 0; i < ST; ++i)
    if (i < mine) load(i, ring + i * STAGE);
  i32x4 acc[NN];
#pragma unroll
  for (int j = 0; j < NN; ++j) acc[j] = i32x4{0, 0, 0, 0};
  int8_t* buf = ring;
  i32x4 fw[2][NN], fx[2];
  auto read = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int8_t* at = buf + 16 * ((4 * h + q) ^ (r & 7)) + r * KS;
      fx[h] = *reinterpret_cast<const i32x4*>(at);
#pragma unroll
      for (int j = 0; j < NN; ++j) fw[h][j] = *reinterpret_cast<const i32x4*>(at + 16 * KS * (1 + j));
    }
    wait_lds();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NN; ++j) acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[h][j], fx[h], acc[j], 0, 0, 0);
    buf = buf + STAGE == ring + ST * STAGE ? ring : buf + STAGE;
  };
  // no branch in this loop, as in the tiles below; then what is left in the ring
  for (int st = 0; st < mine - ST; ++st) {
    wait_vm<(ST - 1) * L>();
    asm volatile("" ::: "memory");
    read();
    load(st + ST, buf);
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
  for (int i = threadIdx.x; i < 16 * NN; i += T) {
    const int n = min(i0 + i % COLS, a.n - 1);
    scales[i] = a.w_scale[((size_t)t.e * P + i / COLS) * a.n + n];
  }
  if (threadIdx.x < 16) scales[16 * NN + threadIdx.x] = a.x_scale[x_row(a, yr[threadIdx.x])];
  __syncthreads();
  // accumulator register c of lane 16 q + r: matrix row 16 j + 4 q + c, row r of x
  int* red = reinterpret_cast<int*>(lds);
#pragma unroll
  for (int j = 0; j < NN; ++j) *reinterpret_cast<i32x4*>(red + (wv * 16 + r) * (16 * NN) + 16 * j + 4 * q) = acc[j];
  __syncthreads();
  for (int i = threadIdx.x; i < t.rows * COLS; i += T) {
    const int m = i / COLS, c = i % COLS;
    if (i0 + c >= a.n) continue;
    float v[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int tc = COLS * p + c;  // column of the tile
      int sum = 0;
#pragma unroll
      for (int w = 0; w < NW; ++w) sum += red[(w * 16 + m) * (16 * NN) + tc];
      v[p] = scaled(sum, scales[16 * NN + m], scales[tc]);
    }
    store_y(a.y, a.y_dtype, (size_t)yr[m] * a.n + i0 + c, P == 2 ? swiglu_f(v[0], v[P - 1]) : v[0]);
  }
}

// One float row of x, quantised on the way: each workgroup finds the row's scale
// and codes itself (14 KB at K 7168, from L2) while the first stages of its 16
// matrix rows travel, which costs less than a launch of its own.  8 waves, so that
// this is short and few stages follow: N 7168, K 7168 10.5 us back to back (4.9 TB/s;
// 4 waves with 32 rows 12.0), N 1536 6.6 (8.7), N 65536 73 (6.4 TB/s).  Grouped: every
// slot reads this row.
constexpr int kTokenBytes = 32768;  // of x at most
constexpr size_t kMaxGroups = ((size_t)1 << 31) / 512;  // workgroups of a launch: its threads, and numbers in int

template <int DT, int P, int NW, int ST>
__global__ __launch_bounds__(64 * NW) void k_i8_token(I8Args a, const u32x4* __restrict__ x, int tiles_n) {
  constexpr int T = 64 * NW, STAGE = 16 * KS, L = 2, COLS = 16 / P, N = Chunk<DT>::N, NC = kTokenBytes / 16 / T;
  __shared__ __attribute__((aligned(1024))) int8_t lds[NW * ST * STAGE];
  __shared__ __attribute__((aligned(16))) int8_t row[kTokenBytes / 16 * N];  // the codes of x
  __shared__ uint32_t part[NW];
  __shared__ __attribute__((aligned(16))) int red[NW][16];
  Tile t;
  if (!find_tile<16>(a, blockIdx.x / tiles_n, t)) return;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i0 = blockIdx.x % tiles_n * COLS, K = a.k, C = K / N;
  if (t.e >= a.num_experts) {  // slots without an expert: rows of zeros
    for (int i = threadIdx.x; i < t.rows * COLS; i += T)
      if (i0 + i % COLS < a.n) store_y(a.y, a.y_dtype, (size_t)y_row(a, t.p0 + i / COLS) * a.n + i0 + i % COLS, 0.0f);
    return;
  }
  u32x4 c[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) c[i] = (int)threadIdx.x + T * i < C ? x[threadIdx.x + T * i] : u32x4{0u, 0u, 0u, 0u};
  __builtin_amdgcn_sched_barrier(0);
  const int lr = lane >> 3, chunk = (lane ^ lr) & 7;
  const int8_t* src[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int n = min(i0 + (P == 2 ? lr : 8 * i + lr), a.n - 1);  // P 2: 8 gate rows, 8 up rows
    src[i] = a.w + (((size_t)t.e * P + (P == 2 ? i : 0)) * a.n + n) * K;
  }
  const int stages = (K + KS - 1) / KS, mine = wv < stages ? (stages - wv + NW - 1) / NW : 0;
  int8_t* ring = lds + wv * ST * STAGE;
  auto load = [&](int i, int8_t* buf) {  // this wave's i-th stage
    const int k = min((wv + NW * i) * KS + 16 * chunk, K - 16);
#pragma unroll
    for (int j = 0; j < L; ++j) load_to_lds<true>(src[j] + k, buf + 1024 * j);
  };
#pragma unroll
  for (int i = 0; i < ST; ++i)
    if (i < mine) load(i, ring + i * STAGE);
  __builtin_amdgcn_sched_barrier(0);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    float v[N];
    Chunk<DT>::widen(c[i], v);
#pragma unroll
    for (int j = 0; j < N; ++j) m = max(m, abs_bits(v[j]));
  }
  m = wave_max_bits(m);
  if (lane == 0) part[wv] = m;
  wait_lds();
  meet();
  m = part[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) m = max(m, part[i]);
  const RowScale rs = row_scale(m);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    // chunks past K, up to the end of its last stage, come out as zeros
    const int at = threadIdx.x + T * i;
    if (at >= stages * (KS / N)) break;
    float v[N];
    Chunk<DT>::widen(c[i], v);
    uint32_t o[N / 4];
    quant_chunk<N>(v, rs, o);
    if constexpr (N == 8) reinterpret_cast<u32x2*>(row)[at] = u32x2{o[0], o[1]};
    else reinterpret_cast<uint32_t*>(row)[at] = o[0];
  }
  wait_lds();
  meet();
  i32x4 acc{0, 0, 0, 0};
  int8_t* buf = ring;
  i32x4 fw[2], fx[2];
  auto read = [&](int st) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      fx[h] = *reinterpret_cast<const i32x4*>(row + (wv + NW * st) * KS + 64 * h + 16 * q);  // the row in all 16 columns
      fw[h] = *reinterpret_cast<const i32x4*>(buf + 16 * ((4 * h + q) ^ (r & 7)) + r * KS);
    }
    wait_lds();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[h], fx[h], acc, 0, 0, 0);
    buf = buf + STAGE == ring + ST * STAGE ? ring : buf + STAGE;
  };
  for (int st = 0; st < mine - ST; ++st) {
    wait_vm<(ST - 1) * L>();
    asm volatile("" ::: "memory");
    read(st);
    load(st + ST, buf);
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
  if (r == 0) *reinterpret_cast<i32x4*>(&red[wv][4 * q]) = acc;
  __syncthreads();
  const int n = i0 + (int)threadIdx.x;
  if ((int)threadIdx.x >= COLS || n >= a.n) return;
  float v[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int tc = threadIdx.x + 8 * p;
    int sum = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += red[w][tc];
    v[p] = scaled(sum, rs.stored, a.w_scale[((size_t)t.e * P + p) * a.n + n]);
  }
  const float y = P == 2 ? swiglu_f(v[0], v[P - 1]) : v[0];
  for (int i = 0; i < t.rows; ++i) store_y(a.y, a.y_dtype, (size_t)y_row(a, t.p0 + i) * a.n + n, y);
}

bool i8_token_ok(const void* x, int dtype, int k, int n, bool swiglu, int max_tiles) {
  const int per = dtype == MOE_DTYPE_F32 ? 4 : 8;  // elements of 16 bytes
  const size_t groups = ((size_t)n * (swiglu ? 2 : 1) + 15) / 16 * max_tiles;
  return reinterpret_cast<uintptr_t>(x) % 16 == 0 && k <= kTokenBytes / 16 * per - KS && groups < kMaxGroups;
}

template <int DT>
static void token_dt(const I8Args& a, const void* x, int max_tiles, hipStream_t s) {
  const int tiles_n = (a.n * (a.swiglu ? 2 : 1) + 15) / 16;
  const dim3 grid(tiles_n * max_tiles), block(512);
  const u32x4* xv = static_cast<const u32x4*>(x);
  if (a.swiglu) hipLaunchKernelGGL((k_i8_token<DT, 2, 8, 3>), grid, block, 0, s, a, xv, tiles_n);
  else hipLaunchKernelGGL((k_i8_token<DT, 1, 8, 3>), grid, block, 0, s, a, xv, tiles_n);
}

hipError_t launch_i8_token(const I8Args& a, const void* x, int dtype, int max_tiles, hipStream_t s) {
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
// into LDS, before stage k is computed.  (Loads through registers instead, of all or
// of the matrix alone, took 12% to 20% longer.)
//
// 256 x 256 tiles: 8192 rows, N 7168, K 7168 take 338 us back to back on the same random
// codes (2.5 POP/s), about 370 behind a quantiser with changing inputs, up to 420 under a profiler,
// and 266 with zeros.  Two bounds lie together, the multiplications of a stage (2048 clocks of the
// matrix units) and its LDS
// traffic (192 KB out and 64 KB in, 2048 clocks at 128 bytes); the counters show the matrix
// units busy for 167 us at 2.4 GHz, and what random codes take more than zeros is the clock
// that the power limit leaves.  At K 1536 a tile takes 28 us: 19 for its 12 stages, 2 to start, 7 for the
// outputs.  (One workgroup a CU that goes from tile to tile, loading the first
// stage of the next one ahead: 8% slower, its waves wait for their own stores.)
// The smaller tiles are bound by the latency of a stage, loads to LDS, barrier, LDS to
// registers, multiplications: 509 rows, SwiGLU of 2 x 1536, K 7168 22 us (1.0 POP/s).

// One tile configuration: BM rows of x by BN matrix rows (P matrices
// interleaved), KG groups of WGM x WGN waves that take the stages in turn, ST
// buffers of a stage.
template <int BM_, int BN_, int WGM_, int WGN_, int KG_, int P_, int ST_>
struct TileCfg {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, KG = KG_, P = P_, ST = ST_;
  static constexpr int NW = WGM * WGN, T = 64 * NW * KG;                     // waves of a group, threads
  static constexpr int MF = BM / WGM / 16, NF = BN / WGN / 16, MO = MF / KG;  // fragments of a wave, rows of them it stores
  static constexpr bool SPLIT = BM == 64 && BN == 64;  // K may be split over workgroups
  static constexpr int STAGE = (BM + BN) * KS, RING = ST * STAGE;
};

// Exchanges between the 16-lane groups of a wave so that of two neighbouring fragments
// (x: columns 4 q .. of the first, y: of the second) lane 16 q + r gets 8 columns from
// 8 q: a store then writes 64 bytes of a row.  (Through LDS, whole rows at a time, the
// outputs of a 256 x 256 tile took 2 us longer: two barriers with nothing beside them.)
__device__ __forceinline__ u32x4 join_fragments(const u32x2& x, const u32x2& y) {
  u32x4 o;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const auto h = __builtin_amdgcn_permlane32_swap(x[k], y[k], false, false);
    const auto f = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
    o[k] = f[0];
    o[2 + k] = f[1];
  }
  return o;
}

// Scales a wave's sums and stores them: its fragment rows from `first` on.  Register
// c of acc[i][j] of lane 16 q + r: matrix row 16 j + 4 q + c, row 16 i + r of x.
template <int DT, class C>
__device__ __forceinline__ void tile_store(const I8Args& a, const Tile& t, const int8_t* lds, int i0, int wm, int wn,
                                           int first, const i32x4 (&acc)[C::MO][C::NF]) {
  constexpr int P = C::P, OB = Elem<DT>::bytes, V = 16 / OB;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const float* sw = reinterpret_cast<const float*>(lds + C::RING);
  const float* sx = sw + C::BN;
  const int* yr = reinterpret_cast<const int*>(sx + C::BM);
  const bool whole = a.n % V == 0;  // 16-byte stores stay aligned, and a chunk is inside the row or outside
  const int c0 = i0 + wn * (C::BN / C::WGN / P);
#pragma unroll
  for (int i = 0; i < C::MO; ++i) {
    const int m = 16 * (C::WGM * (first + i) + wm) + r;
    if (m - r >= t.rows) break;
    const float s = sx[m];
    const size_t row = (size_t)yr[m] * a.n;
    // Gates below -80 are rare: the row is stored as if there were none, and once more if
    // there are.  (A branch for each value took 8192 rows of 2 x 3584, K 1536 from 122 to
    // 127.5 us, one for each fragment to 123.4.)
    float lowest = 0.0f;
    auto values = [&](int j, auto low) {  // of output fragment j
      f32x4 v;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const f32x4 w = *reinterpret_cast<const f32x4*>(sw + (wn * C::NF + j * P + p) * 16 + 4 * q);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float u = scaled(acc[i][j * P + p][c], s, w[c]);
          if (p) lowest = fminf(lowest, v[c]);
          v[c] = !p ? u : decltype(low)::value ? swiglu_f(v[c], u) : swiglu_rest(v[c], u);
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
__device__ __forceinline__ void tile_store_part(const I8Args& a, const Tile& t, int tn, int tiles_n, int wm, int wn,
                                                int part, int first, const i32x4 (&acc)[C::MO][C::NF]) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const size_t width = (size_t)tiles_n * C::BN;
  int* dst = a.parts + ((size_t)part * a.rows + t.p0) * width + tn * C::BN + wn * C::NF * 16 + 4 * q;
#pragma unroll
  for (int i = 0; i < C::MO; ++i) {
    const int m = 16 * (C::WGM * (first + i) + wm) + r;
    if (m >= t.rows) continue;
#pragma unroll
    for (int j = 0; j < C::NF; ++j) *reinterpret_cast<i32x4*>(dst + m * width + 16 * j) = acc[i][j];
  }
}

// The end of a tile: its outputs, or its part of the sums.
template <class C>
__device__ __forceinline__ void tile_end(const I8Args& a, const Tile& t, const int8_t* lds, int i0, int tn, int tiles_n,
                                         int wm, int wn, int parts, int part, int first,
                                         const i32x4 (&acc)[C::MO][C::NF]) {
  if constexpr (C::SPLIT) {
    if (parts > 1) {
      tile_store_part<C>(a, t, tn, tiles_n, wm, wn, part, first, acc);
      return;
    }
  }
  if (a.y_dtype == MOE_DTYPE_BF16) tile_store<MOE_DTYPE_BF16, C>(a, t, lds, i0, wm, wn, first, acc);
  else if (a.y_dtype == MOE_DTYPE_F16) tile_store<MOE_DTYPE_F16, C>(a, t, lds, i0, wm, wn, first, acc);
  else tile_store<MOE_DTYPE_F32, C>(a, t, lds, i0, wm, wn, first, acc);
}

template <class C>
__global__ __launch_bounds__(C::T) void k_i8_tile(I8Args a, int tiles_n, int tiles_m, int parts, int band_rows) {
  constexpr int BM = C::BM, BN = C::BN, WGM = C::WGM, WGN = C::WGN, P = C::P, ST = C::ST, NW = C::NW, MF = C::MF,
                KG = C::KG, NF = C::NF, GX = BM / 8, L = (BM + BN) / 8 / NW;  // L: loads of a wave and stage
  static_assert(L * 8 * NW == BM + BN && NF % P == 0 && ST % KG == 0 && GX == NW * MF &&
                    (KG == 1 || NW == 4), "tile");
  // the ring, then the tile's matrix scales, row scales and output rows
  __shared__ __attribute__((aligned(1024))) int8_t lds[C::RING + 4 * (BN + 2 * BM)];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), kg = wave / NW, wv = wave % NW;
  const int wm = wv % WGM, wn = wv / WGM;
  // a grouped product's grid is sized for the most tiles its slots can make: the
  // XCDs share the ones there are
  const TileAt at = tile_at(blockIdx.x, tiles_n, tiles_m, a.order ? a.num_tiles[0] : tiles_m, parts, band_rows);
  if (!at.any) return;
  const int tn = at.tn, tm = at.tm, part = at.part;
  Tile t;
  if (!find_tile<BM>(a, tm, t)) return;
  const int K = a.k, i0 = tn * (BN / P);  // first output column
  if (t.e >= a.num_experts) {
    for (int m = wave; m < t.rows; m += KG * NW)
      for (int n = i0 + lane; n < min(i0 + BN / P, a.n); n += 64)
        store_y(a.y, a.y_dtype, (size_t)y_row(a, t.p0 + m) * a.n + n, 0.0f);
    return;
  }
  float* scales = reinterpret_cast<float*>(lds + C::RING);
  int* yr = reinterpret_cast<int*>(scales + BN + BM);
  for (int i = threadIdx.x; i < BM; i += C::T) yr[i] = y_row(a, t.p0 + min(i, t.rows - 1));
  __syncthreads();
  // Loads: a wave copies 8 rows x 128 codes at a time; lane l brings chunk
  // (l ^ row) & 7 of row l >> 3, so that the same 16-byte chunk of 8 consecutive
  // rows lies in 8 different bank groups when a fragment reads it.
  const int lr = lane >> 3, chunk = (lane ^ lr) & 7;
  const int8_t* src[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int g = wv + NW * i;  // group of 8 rows: first those of x, then the matrix's
    if (g < GX) {
      src[i] = a.x + (size_t)x_row(a, yr[8 * g + lr]) * a.x_stride;
    } else {
      const int gw = 8 * (g - GX);  // first row of the tile's matrix part; P 2: 16 gate rows, 16 up rows, ...
      const int n = min(i0 + (P == 2 ? gw / 32 * 16 + gw % 16 : gw) + lr, a.n - 1);
      src[i] = a.w + (((size_t)t.e * P + (P == 2 ? gw / 16 % 2 : 0)) * a.n + n) * K;
    }
  }
  const int stages = (K + KS - 1) / KS;
  const int s0 = (int)((size_t)stages * part / parts), S = (int)((size_t)stages * (part + 1) / parts);
  i32x4 acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  // With U of the MF fragment rows: a tile whose last rows are missing (the end of an
  // expert) neither loads nor multiplies them.
  auto run = [&](auto used) {
    constexpr int U = decltype(used)::value, LU = L - MF + U;
    auto load_whole = [&](int st, int b) {
      int8_t* buf = lds + b * C::STAGE;
#pragma unroll
      for (int i = 0; i < L; ++i)
        if (i < U || i >= MF) load_to_lds(src[i] + (st * KS + 16 * chunk), buf + 1024 * (wv + NW * i));
    };
    auto load = [&](int st, int b) {  // stage st to buffer b
      if ((st + 1) * KS <= K) {
        load_whole(st, b);
      } else {  // the last stage of a K that is no multiple of 128: zeros past K on x's side
        int8_t* buf = lds + b * C::STAGE;
        const int k = st * KS + 16 * chunk;
#pragma unroll
        for (int i = 0; i < L; ++i)
          if (i < U || i >= MF)
            load_to_lds(i < MF && k >= K ? kZeroCodes : src[i] + min(k, K - 16), buf + 1024 * (wv + NW * i));
      }
    };
#pragma unroll
    for (int i = 0; i < ST / KG - 1; ++i)
      if (s0 + KG * i + kg < S) load(s0 + KG * i + kg, KG * i + kg);
    // the scales travel with the first stage; the loop's barriers stand before their use
    for (int i = threadIdx.x; i < BN; i += C::T) {
      const int n = min(i0 + (P == 2 ? i / 32 * 16 + i % 16 : i), a.n - 1);
      scales[i] = a.w_scale[((size_t)t.e * P + (P == 2 ? i / 16 % 2 : 0)) * a.n + n];
    }
    for (int i = threadIdx.x; i < BM; i += C::T) scales[BN + i] = a.x_scale[x_row(a, yr[i])];
    i32x4 fw[NF], fx[U];
    auto read = [&](int b, int half) {
      const int at = 16 * ((4 * half + q) ^ (r & 7)) + r * KS;
      const int8_t* bx = lds + b * C::STAGE + 16 * wm * KS + at;
      const int8_t* bw = lds + b * C::STAGE + BM * KS + wn * (BN / WGN) * KS + at;
#pragma unroll
      for (int j = 0; j < NF; ++j) fw[j] = *reinterpret_cast<const i32x4*>(bw + 16 * KS * j);
#pragma unroll
      for (int i = 0; i < U; ++i) fx[i] = *reinterpret_cast<const i32x4*>(bx + 16 * WGM * KS * i);
    };
    auto multiply = [&]() {
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[j], fx[i], acc[i][j], 0, 0, 0);
    };
    // waits until all loads of this wave but those of the `later` newest stages have landed
    auto landed = [&](int later) {
      if (later >= 2) wait_vm<2 * LU>();
      else if (later == 1) wait_vm<LU>();
      else wait_vm<0>();
    };
    // Stages whose own load is a whole one go first, in a loop without a branch (each
    // costs tens of clocks, and a stage of a small tile is a few hundred).
    int i = 0;
    const int n = S - s0;  // stage s0 + i is in buffer i
    if constexpr (NW == 8) {
      // Two waves a SIMD, of two groups one step apart: while the waves of one
      // group multiply, those of the other read the fragments of half a stage from
      // LDS and issue loads, then they change places at a barrier.  A stage has
      // landed for every wave when a group reads it: each wave waited for its own
      // loads of the next stage before the barrier that ends its reads of this one.
      const bool second = wv >= 4;
      landed(min(ST - 2, n - 1));
      meet();
      if (second) meet();
      auto turn = [&]() {
        meet();
        __builtin_amdgcn_s_setprio(1);
        multiply();
        __builtin_amdgcn_s_setprio(0);
        meet();
      };
      for (; i < n - ST; ++i) {
        read(i & (ST - 1), 0);
        load_whole(s0 + i + ST - 1, (i + ST - 1) & (ST - 1));  // both groups have read stage i - 1
        wait_lds();
        turn();
        read(i & (ST - 1), 1);
        wait_vm<(ST - 2) * LU>();
        turn();
      }
      for (; i < n; ++i) {
        read(i & (ST - 1), 0);
        if (i + ST - 1 < n) load(s0 + i + ST - 1, (i + ST - 1) & (ST - 1));
        wait_lds();
        turn();
        read(i & (ST - 1), 1);
        landed(min(ST - 2, n - 2 - i));
        turn();
      }
      if (!second) meet();
    } else {
      // One or two groups of four waves: while one reads fragments, the other multiplies.  Group kg
      // has stages kg, kg + KG, ... and loads them itself; at the barrier of turn i every group has
      // its stage of that turn, and has left the buffer of the turn before.  (One group of four
      // waves: 19 us where two take 15.7, 128 rows, N 7168, K 7168.)  A ring is one body, so that
      // its buffers are constants: with their numbers in registers 64 x 128 tiles took 30 us for 21.
      constexpr int R = ST / KG;
      auto multiply_stage = [&](int b) {
        read(b, 0);
        multiply();
        read(b, 1);
        multiply();
      };
      const int mine = (n - kg + KG - 1) / KG, turns = (n + KG - 1) / KG;
      for (; i <= turns - 2 * R; i += R) {
#pragma unroll
        for (int u = 0; u < R; ++u) {
          wait_vm<(R - 2) * LU>();
          meet();
          load_whole(s0 + KG * (i + u + R - 1) + kg, KG * ((u + R - 1) % R) + kg);
          multiply_stage(KG * u + kg);
        }
      }
#pragma unroll
      for (int u = 0; u < 2 * R - 1; ++u) {
        if (i + u >= turns) break;
        landed(min(R - 2, mine - 1 - i - u));
        meet();
        if (i + u + R - 1 < mine) load(s0 + KG * (i + u + R - 1) + kg, KG * ((u + R - 1) % R) + kg);
        if (i + u < mine) multiply_stage(KG * (u % R) + kg);
      }
    }
  };
  const int need = (t.rows + 16 * WGM - 1) / (16 * WGM);
  if (need >= MF) run(std::integral_constant<int, MF>{});
  else if (MF == 4 && need == 3) run(std::integral_constant<int, MF == 4 ? 3 : 1>{});
  else if (MF == 4 && need == 2) run(std::integral_constant<int, MF == 4 ? 2 : 1>{});
  else run(std::integral_constant<int, 1>{});
  if constexpr (KG == 1) {
    tile_end<C>(a, t, lds, i0, tn, tiles_n, wm, wn, parts, part, 0, acc);
  } else {
    // each group gives the other half of its fragment rows away and adds what it gets
    i32x4* swap = reinterpret_cast<i32x4*>(lds) + (wv * C::MO * NF) * 64 + lane;
    constexpr int HALF = NW * C::MO * NF * 64;
    static_assert(2 * HALF * 16 <= C::RING, "sums");
    i32x4 sum[C::MO][NF];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < C::MO; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        sum[i][j] = kg ? acc[C::MO + i][j] : acc[i][j];
        swap[kg * HALF + (i * NF + j) * 64] = kg ? acc[i][j] : acc[C::MO + i][j];
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < C::MO; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) sum[i][j] += swap[(1 - kg) * HALF + (i * NF + j) * 64];
    tile_end<C>(a, t, lds, i0, tn, tiles_n, wm, wn, parts, part, kg * C::MO, sum);
  }
}

constexpr int kMaxParts = 8;

// The parts of a split K (of a dense product) added up, scaled and stored: a
// workgroup takes 4 rows, a wave each, by 256 columns.
template <class C>
__global__ __launch_bounds__(256) void k_i8_parts(I8Args a, int parts, int tiles_n, int cols) {
  constexpr int P = C::P, BO = C::BN / P;
  const int m = blockIdx.x / cols * 4 + (threadIdx.x >> 6), n = blockIdx.x % cols * 256 + (threadIdx.x & 63) * 4;
  if (m >= a.rows || n >= a.n) return;
  const float sx = a.x_scale[m];
  const float* sw = a.w_scale;
  const size_t width = (size_t)tiles_n * C::BN, step = (size_t)a.rows * width;
  const int* src = a.parts + (size_t)m * width + n / BO * C::BN + n % BO / 16 * 16 * P + n % 16;
  float v[P][4];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    i32x4 sum{0, 0, 0, 0}, part[kMaxParts];  // all parts requested before the first is added
#pragma unroll
    for (int i = 0; i < kMaxParts; ++i)
      part[i] = *reinterpret_cast<const i32x4*>(src + min(i, parts - 1) * step + 16 * p);
#pragma unroll
    for (int i = 0; i < kMaxParts; ++i) sum += i < parts ? part[i] : i32x4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) v[p][k] = scaled(sum[k], sx, sw[p * a.n + min(n + k, a.n - 1)]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (P == 2) v[0][k] = swiglu_f(v[0][k], v[P - 1][k]);
    if (n + k < a.n) store_y(a.y, a.y_dtype, (size_t)m * a.n + n + k, v[0][k]);
  }
}

template <class C>
static void tile_launch(const I8Args& a, int max_tiles, int parts, hipStream_t s) {
  const int tiles_n = (a.n * C::P + C::BN - 1) / C::BN;
  const int per_xcd = (tiles_n * max_tiles * parts + 7) / 8;
  int band = 8;
  if (a.order) {
    band = (a.rows / a.num_experts + C::BM / 2) / C::BM;
    band = band < 1 ? 1 : band > 8 ? 8 : band;
  }
  hipLaunchKernelGGL(k_i8_tile<C>, dim3(8 * per_xcd), dim3(C::T), 0, s, a, tiles_n, max_tiles, parts, band);
  if constexpr (C::SPLIT) {
    if (parts == 1) return;
    const int cols = (a.n + 255) / 256;
    hipLaunchKernelGGL(k_i8_parts<C>, dim3(cols * ((a.rows + 3) / 4)), dim3(256), 0, s, a, parts, tiles_n, cols);
  }
}

// 32 matrix rows a workgroup, or 16 where all those have a CU to themselves (8 rows,
// SwiGLU of 2 x 1536, K 7168: 6.7 us for 8.7; 37 rows, N 1536, 288 of them: 9.3 for 8.2).
static void stream_launch(const I8Args& a, int max_tiles, hipStream_t s) {
  const int rows = a.n * (a.swiglu ? 2 : 1), halves = (rows + 15) / 16;
  const dim3 block(256);
  if (halves * max_tiles <= 256) {
    if (a.swiglu) hipLaunchKernelGGL((k_i8_stream<1, 2, 4, 3>), dim3(halves * max_tiles), block, 0, s, a, halves);
    else hipLaunchKernelGGL((k_i8_stream<1, 1, 4, 3>), dim3(halves * max_tiles), block, 0, s, a, halves);
    return;
  }
  const int tiles_n = (rows + 31) / 32;
  if (a.swiglu) hipLaunchKernelGGL((k_i8_stream<2, 2, 4, 2>), dim3(tiles_n * max_tiles), block, 0, s, a, tiles_n);
  else hipLaunchKernelGGL((k_i8_stream<2, 1, 4, 2>), dim3(tiles_n * max_tiles), block, 0, s, a, tiles_n);
}

// The kernels a product may run on, in the order of I8Plan::kind: 16 rows of x by 32
// matrix rows as a stream, and the tiles.
struct Tiling {
  int bm, bn;
  int resident;            // workgroups that the card holds at a time
  bool rounds;             // dense: time goes by whole rounds of them
  double d0, d1;           // dense: us a round, and a stage of a round
  double g0, g1, g2, g3, g4;  // grouped, see i8_plan
};
constexpr Tiling kTilings[] = {{16, 32, 512, false, 3.3, 0.105, 3.9, 0.88, 0.257, 0.0, 0.06},
                               {64, 64, 256, true, 3.0, 0.21, 0.4, 2.9, 0.118, 0.106, 0.422},
                               {64, 128, 256, true, 4.0, 0.30, 0.0, 3.46, 0.173, 0.136, 0.549},
                               {128, 128, 256, true, 4.5, 0.54, 0.0, 4.58, 0.118, 0.379, 0.354},
                               {128, 128, 512, false, 6.1, 1.15, 0.0, 4.99, 0.569, 0.0, 0.49},
                               {256, 256, 256, true, 7.0, 1.4, 0.0, 6.44, 0.869, 0.0, 0.453}};
constexpr int kStream = 0, kSplit = 1, kTwoToACu = 4;

// Which kernel a product runs on: the one with the least estimated time.
// Dense: T workgroups in rounds of those that the card holds, each d0 + d1 * stages.  Up
// to 16 rows always the stream; with more rows it reads the matrix again for every 16, and is
// taken where all its workgroups get a CU to themselves.  Two 128 x 128 tiles to a CU (two
// buffers of a stage each) are for more than one round of single ones (four buffers).
// Measured at N 7168, K 7168: 8 rows 10.2 us (64 x 64 tiles 12.0), 24 rows 18.4 (12.4); 128 rows:
// 64 x 64 15.8 us, 64 x 128 20.4, 128 x 128 30.8; 500 rows: 55, 41, 37, 256 x 256 68; 2048 rows: 191,
// 145, 136 (two to a CU: 108), 86.  Over 110 products of 17 to 4096 rows, N 128 to 8192, K 128 to
// 8192 the choice costs 1.6% over the best kernel on average and 9% in the worst tenth: short K
// with some 30 to 200 rows, where the stream would take 1 to 2 us less (97 rows, 2 x 268, K 176: 6.0 us, 4.0).
// Grouped: each expert's matrix comes from HBM, an expert's rows end anywhere in a tile
// (half a tile more on average, of which only the rows that there are cost anything).
// g0 + rounds * (g1 + g2 * stages) + g3 * stages * rounds' worth of rows + g4 * the time to read
// the matrices at 6.6 TB/s, fitted to 165 products of 4 to 256 experts with 2 to 500
// rows each, K 768 to 7168: the choice costs 3% over the best kernel on average.  16
// experts, N 4096, K 4096, 80 rows each: 64 x 64 96 us, 128 x 128 65 (two to a CU: 50), 256 x
// 256 56; 320 rows: 236, 132, 127, 119.  128 experts of 12 rows, N 2048, K 768: the stream 53
// us, 128 x 128 39; 32 experts of 8, 2 x 1536, K 7168: 111, 151.
// K is split over parts where 64 x 64 tiles leave most CUs without work and the stages saved
// are worth adding the parts up, 5 us and more (64 rows of N 1536, K 7168: 10.4 us in 8
// parts, 11.5 in one; 24 rows of N 7168: 14.6 in 2 parts, 12.2 in one).
I8Plan i8_plan(int rows, int experts, bool grouped, int n, int k, bool swiglu) {
  const int P = swiglu ? 2 : 1, stages = (k + KS - 1) / KS, used = !grouped ? 1 : rows < experts ? rows : experts;
  const double per = (double)rows / used, read = (double)used * n * P * k / 6.6e6;
  I8Plan best{-1, 0, 1, 0};
  double least = 0.0;
  for (int kind = 0; kind < (int)(sizeof(kTilings) / sizeof(kTilings[0])); ++kind) {
    const Tiling& m = kTilings[kind];
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
      if (kind == kStream ? rows > 16 && tiles > 256.0 : kind == kTwoToACu && tiles <= 256.0) continue;
      double load = m.rounds ? ceil(tiles / m.resident) : tiles / m.resident;
      if (load < 1.0) load = 1.0;
      time = kind == kStream && rows <= 16 ? 0.0 : (m.d0 + m.d1 * stages) * load;
      if (kind == kSplit) {
        parts = (int)(224.0 / tiles);
        if (parts > kMaxParts) parts = kMaxParts;
        if (parts > stages / 6) parts = stages / 6;
        const double saved = parts > 1 ? m.d1 * (stages - stages / parts) - 8.0 : 0.0;
        if (saved <= 0.0) parts = 1;
        else time -= saved;
      }
    }
    if (best.kind >= 0 && time >= least) continue;
    least = time;
    best = I8Plan{kind, m.bm, parts, parts > 1 ? (size_t)parts * rows * cols * m.bn * 4 : 0};
  }
  return best;
}

template <int P>
static void tiles_launch(const I8Args& a, const I8Plan& plan, int max_tiles, hipStream_t s) {
  if (plan.kind == 1) tile_launch<TileCfg<64, 64, 2, 2, 2, P, 8>>(a, max_tiles, plan.parts, s);
  else if (plan.kind == 2) tile_launch<TileCfg<64, 128, 2, 2, 2, P, 6>>(a, max_tiles, 1, s);
  else if (plan.kind == 3) tile_launch<TileCfg<128, 128, 4, 2, 1, P, 4>>(a, max_tiles, 1, s);
  else if (plan.kind == 4) tile_launch<TileCfg<128, 128, 4, 2, 1, P, 2>>(a, max_tiles, 1, s);
  else tile_launch<TileCfg<256, 256, 4, 2, 1, P, 2>>(a, max_tiles, 1, s);
}

bool i8_launchable(const I8Plan& plan, int n, bool swiglu, int max_tiles) {
  const size_t bn = kTilings[plan.kind].bn, cols = ((size_t)n * (swiglu ? 2 : 1) + bn - 1) / bn;
  return cols * max_tiles * plan.parts < kMaxGroups;
}

hipError_t launch_gemm_i8(const I8Args& a, const I8Plan& plan, int max_tiles, hipStream_t s) {
  if (plan.kind == 0) stream_launch(a, max_tiles, s);
  else if (a.swiglu) tiles_launch<2>(a, plan, max_tiles, s);
  else tiles_launch<1>(a, plan, max_tiles, s);
  return hipGetLastError();
}

}  // namespace moe
