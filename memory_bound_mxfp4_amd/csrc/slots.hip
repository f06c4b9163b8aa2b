// slots.hip -- the slots of a routing sorted by expert, and the gated sum of
// the experts' outputs.
#include "i8_common.h"

namespace moe {

GroupsLayout groups_layout(int tokens, int top_k, int E) {
  GroupsLayout g;
  const size_t slots = (size_t)tokens * top_k;
  size_t o = align256(4 * slots);
  g.offsets = o;
  o += align256(4 * ((size_t)E + 2));
  g.counts = o;
  o += 256;
  for (int i = 0; i < kTileMaps; ++i) {
    g.tiles[i] = o;
    const size_t partial = slots < (size_t)E + 1 ? slots : (size_t)E + 1;
    g.max_tiles[i] = (int)(slots / kTileRows[i] + partial);
    o += align256(8 * (size_t)g.max_tiles[i]);
  }
  g.bytes = o;
  return g;
}

// Lanes of the wave that hold the same key (of `bits` bits) as this one.
__device__ __forceinline__ uint64_t same_key(int key, int bits, uint64_t active) {
  uint64_t m = active;
  for (int b = 0; b < bits; ++b) {
    const uint64_t bal = __ballot((key >> b) & 1);
    m &= ((key >> b) & 1) ? bal : ~bal;
  }
  return m;
}

// Exclusive sum over the 1024 threads of a block; *total gets the whole.
template <int W>
__device__ __forceinline__ int block_scan(int v, int* part, int* total) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(s, d, WAVE);
    if (lane >= d) s += u;
  }
  __syncthreads();
  if (lane == 63) part[wv] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int p = part[i];
    before += i < wv ? p : 0;
    all += p;
  }
  *total = all;
  return before + s - v;
}

// A stable counting sort by one workgroup.  Each of the W waves owns a
// contiguous range of slots and a row of counters, so a slot's place is its
// expert's first place + the counts of earlier waves + its rank within the
// wave: no atomics, and the order is the same on every run.
template <int W, int EMAX>
__global__ __launch_bounds__(64 * W) void k_group_slots(const int32_t* __restrict__ idx, int slots, int E,
                                                        int32_t* __restrict__ order, int32_t* __restrict__ offsets,
                                                        int32_t* __restrict__ counts, TileMaps maps) {
  __shared__ int cnt[W][EMAX + 1];
  __shared__ int part[W];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < W * (EMAX + 1); i += 64 * W) (&cnt[0][0])[i] = 0;
  __syncthreads();
  const int bits = 32 - __clz(E);  // keys 0 .. E, E: no expert
  const int per = ((slots + W - 1) / W + 63) / 64 * 64;
  const int s0 = min(wv * per, slots), s1 = min(s0 + per, slots);
  for (int b = s0; b < s1; b += 64) {
    const int s = b + lane;
    int e = s < s1 ? idx[s] : E;
    e = (unsigned)e < (unsigned)E ? e : E;
    const uint64_t m = same_key(e, bits, __ballot(s < s1));
    if (s < s1 && (m & ((1ull << lane) - 1)) == 0) cnt[wv][e] += __popcll(m);
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  // the experts' totals, their offsets, and the counters turned into places
  constexpr int EPT = (EMAX + 1 + 64 * W - 1) / (64 * W);
  int tot[EPT], sum = 0;
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    const int e = threadIdx.x * EPT + i;
    tot[i] = 0;
    if (e <= E)
      for (int w = 0; w < W; ++w) tot[i] += cnt[w][e];
    sum += tot[i];
  }
  int all;
  int at = block_scan<W>(sum, part, &all);
  if (threadIdx.x == 0) offsets[E + 1] = slots;
  int first[EPT];
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    const int e = threadIdx.x * EPT + i;
    first[i] = at;
    if (e <= E) {
      offsets[e] = at;
      int run = at;
      for (int w = 0; w < W; ++w) {
        const int c = cnt[w][e];
        cnt[w][e] = run;
        run += c;
      }
    }
    at += tot[i];
  }
#pragma unroll
  for (int k = 0; k < kTileMaps; ++k) {
    const int bm = kTileRows[k];
    int n = 0;
#pragma unroll
    for (int i = 0; i < EPT; ++i) n += (tot[i] + bm - 1) / bm;
    int whole;
    int o = block_scan<W>(n, part, &whole);
    if (threadIdx.x == 0) counts[k] = whole;
#pragma unroll
    for (int i = 0; i < EPT; ++i)
      for (int p = 0; p < tot[i]; p += bm) maps.t[k][o++] = int2{(int)threadIdx.x * EPT + i, first[i] + p};
  }
  __syncthreads();
  for (int b = s0; b < s1; b += 64) {
    const int s = b + lane;
    int e = s < s1 ? idx[s] : E;
    e = (unsigned)e < (unsigned)E ? e : E;
    const uint64_t m = same_key(e, bits, __ballot(s < s1));
    const int rank = __popcll(m & ((1ull << lane) - 1));
    const int base = s < s1 ? cnt[wv][e] : 0;
    __builtin_amdgcn_wave_barrier();
    if (s < s1) {
      order[base + rank] = s;
      if (rank == 0) cnt[wv][e] = base + __popcll(m);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

hipError_t launch_group_slots(const int32_t* idx, int tokens, int top_k, int E, void* groups, hipStream_t s) {
  const GroupsLayout g = groups_layout(tokens, top_k, E);
  char* p = static_cast<char*>(groups);
  TileMaps maps;
  for (int i = 0; i < kTileMaps; ++i) maps.t[i] = reinterpret_cast<int2*>(p + g.tiles[i]);
  int32_t* order = reinterpret_cast<int32_t*>(p);
  int32_t* offsets = reinterpret_cast<int32_t*>(p + g.offsets);
  int32_t* counts = reinterpret_cast<int32_t*>(p + g.counts);
  if (E <= 1024)
    hipLaunchKernelGGL((k_group_slots<16, 1024>), dim3(1), dim3(1024), 0, s, idx, tokens * top_k, E, order, offsets,
                       counts, maps);
  else
    hipLaunchKernelGGL((k_group_slots<8, MOE_MAX_EXPERTS>), dim3(1), dim3(512), 0, s, idx, tokens * top_k, E, order,
                       offsets, counts, maps);
  return hipGetLastError();
}

// out[t] = sum_j gate[t][j] y[t k + j] (j ascending), + residual[t].
template <int DT>
__global__ __launch_bounds__(256) void k_combine(const void* __restrict__ y, const float* __restrict__ gate, int top_k,
                                                 int H, const float* residual, float* out) {
  const size_t t = blockIdx.y;
  const int h = blockIdx.x * 256 + threadIdx.x;
  if (h >= H) return;
  float acc = 0.0f;
  for (int j = 0; j < top_k; ++j) acc = fmaf(gate[t * top_k + j], load_f32<DT>(y, (t * top_k + j) * H + h), acc);
  out[t * H + h] = residual ? residual[t * H + h] + acc : acc;
}

hipError_t launch_combine(const void* y, int dtype, const float* gate, int tokens, int top_k, int H,
                          const float* residual, float* out, hipStream_t s) {
  const int step = 65535;  // grid.y limit
  for (int t0 = 0; t0 < tokens; t0 += step) {
    const int nt = tokens - t0 < step ? tokens - t0 : step;
    const size_t es = dtype == MOE_DTYPE_F32 ? 4 : 2;
    const void* yp = static_cast<const char*>(y) + (size_t)t0 * top_k * H * es;
    const float* gp = gate + (size_t)t0 * top_k;
    const float* rp = residual ? residual + (size_t)t0 * H : nullptr;
    float* op = out + (size_t)t0 * H;
    const dim3 grid((H + 255) / 256, nt), block(256);
    if (dtype == MOE_DTYPE_BF16)
      hipLaunchKernelGGL(k_combine<MOE_DTYPE_BF16>, grid, block, 0, s, yp, gp, top_k, H, rp, op);
    else if (dtype == MOE_DTYPE_F16)
      hipLaunchKernelGGL(k_combine<MOE_DTYPE_F16>, grid, block, 0, s, yp, gp, top_k, H, rp, op);
    else
      hipLaunchKernelGGL(k_combine<MOE_DTYPE_F32>, grid, block, 0, s, yp, gp, top_k, H, rp, op);
  }
  return hipGetLastError();
}

}  // namespace moe
