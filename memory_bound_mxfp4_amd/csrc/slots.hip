// slots.hip -- the slots of a routing sorted by expert, and the gated sum of
// the experts' outputs.
#include "i8_common.h"

namespace moe {

// Slots that one workgroup sorts: 4 rounds of 64 for each of 4 waves, held in
// registers.  (With 16 waves a workgroup the two launches of 32768 slots took 7 and
// 18 us.)
static constexpr int kOneBlock = 1024;

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
  // workgroups of the sort: one up to kOneBlock slots, then one for that many, at most 64
  const size_t blocks = (slots + kOneBlock - 1) / kOneBlock;
  g.blocks = blocks < 64 ? (int)blocks : 64;
  g.hist = o;
  if (g.blocks > 1) o += align256(4 * ((size_t)E + 1) * g.blocks);
  g.bytes = o;
  return g;
}

// Lanes of the wave that hold the same key (of BITS bits) as this one.
template <int BITS>
__device__ __forceinline__ uint64_t same_key(int key, uint64_t active) {
  uint64_t m = active;
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const uint64_t bal = __ballot((key >> b) & 1);
    m &= ((key >> b) & 1) ? bal : ~bal;
  }
  return m;
}

// Exclusive sums over the W waves of a block of NV values a thread; total[]
// gets the whole sums.
template <int W, int NV>
__device__ __forceinline__ void block_scan(const int (&v)[NV], int (&before)[NV], int (&total)[NV], int (*part)[NV]) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int s[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) s[k] = v[k];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1)
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int u = __shfl_up(s[k], d, WAVE);
      if (lane >= d) s[k] += u;
    }
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (lane == 63) part[wv][k] = s[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    before[k] = s[k] - v[k];
    total[k] = 0;
  }
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int p = part[i][k];
      before[k] += i < wv ? p : 0;
      total[k] += p;
    }
}

// A stable counting sort.  Each wave owns a contiguous range of slots and a
// row of counters in LDS, so a slot's place is its expert's first place + the
// counts of earlier waves + its rank within the wave: no atomics, and the
// order is the same on every run.  A wave holds R x 64 experts in registers
// between counting and placing; longer ranges are read twice.
//
// One workgroup does it all up to kOneBlock slots.  Above that a first launch
// (PHASE 1) counts each block's slots per expert into hist[block][E + 1], and a
// second one (PHASE 2) adds up the blocks before its own and places.  Bound by
// latency: 128 slots of 128 experts 4.8 us, 32768 of 64 in two launches 5.2 and 8.9.
template <int W, int EMAX, int PHASE>
__global__ __launch_bounds__(64 * W) void k_group_slots(const int32_t* __restrict__ idx, int slots, int per_block,
                                                        int E, int32_t* __restrict__ order,
                                                        int32_t* __restrict__ offsets, int32_t* __restrict__ counts,
                                                        int32_t* __restrict__ hist, TileMaps maps) {
  constexpr int R = 4, NV = 1 + kTileMaps, BITS = EMAX <= 1024 ? 11 : 13;  // keys 0 .. E, E: no expert
  __shared__ int cnt[W * (EMAX + 1)];
  __shared__ int part[W][NV];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, E1 = E + 1;
  int* mine = cnt + wv * E1;
  for (int i = threadIdx.x; i < W * E1; i += 64 * W) cnt[i] = 0;
  const int b0 = min((int)blockIdx.x * per_block, slots), b1 = min(b0 + per_block, slots);
  const int per = ((b1 - b0 + W - 1) / W + 63) / 64 * 64;
  const int s0 = min(b0 + wv * per, b1), s1 = min(s0 + per, b1);
  int key[R];
  uint64_t same[R];
  auto fetch = [&](int b) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int s = b + 64 * i + lane;
      const int e = s < s1 ? idx[s] : E;
      key[i] = (unsigned)e < (unsigned)E ? e : E;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) same[i] = same_key<BITS>(key[i], __ballot(b + 64 * i + lane < s1));
  };
  fetch(s0);
  __syncthreads();
  for (int b = s0; b < s1; b += 64 * R) {
    if (b > s0) fetch(b);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (b + 64 * i + lane < s1 && (same[i] & ((1ull << lane) - 1)) == 0) mine[key[i]] += __popcll(same[i]);
      wave_sync();
    }
  }
  __syncthreads();
  if (PHASE == 1) {
    for (int e = threadIdx.x; e < E1; e += 64 * W) {
      int t = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) t += cnt[w * E1 + e];
      hist[(size_t)blockIdx.x * E1 + e] = t;
    }
    return;
  }
  // the experts' totals, their first places, and the counters turned into places
  constexpr int EPT = (EMAX + 1 + 64 * W - 1) / (64 * W);
  const int ept = (E1 + 64 * W - 1) / (64 * W);
  int tot[EPT], ahead[EPT], v[NV], at[NV], all[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) v[k] = 0;
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    const int e = threadIdx.x * ept + i;
    tot[i] = ahead[i] = 0;
    if (i < ept && e < E1) {
      if (PHASE == 2) {
        for (int g = 0; g < (int)gridDim.x; g += 8) {  // eight loads at a time
          int c[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) c[u] = hist[(size_t)min(g + u, (int)gridDim.x - 1) * E1 + e];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            tot[i] += g + u < (int)gridDim.x ? c[u] : 0;
            ahead[i] += g + u < (int)blockIdx.x ? c[u] : 0;
          }
        }
      } else {
#pragma unroll
        for (int w = 0; w < W; ++w) tot[i] += cnt[w * E1 + e];
      }
    }
    v[0] += tot[i];
#pragma unroll
    for (int k = 0; k < kTileMaps; ++k) v[1 + k] += (tot[i] + kTileRows[k] - 1) / kTileRows[k];
  }
  block_scan<W, NV>(v, at, all, part);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    offsets[E1] = slots;
#pragma unroll
    for (int k = 0; k < kTileMaps; ++k) counts[k] = all[1 + k];
  }
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    const int e = threadIdx.x * ept + i;
    if (i < ept && e < E1) {
      int run = at[0] + ahead[i], c[W];
#pragma unroll
      for (int w = 0; w < W; ++w) c[w] = cnt[w * E1 + e];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        cnt[w * E1 + e] = run;
        run += c[w];
      }
      if (blockIdx.x == 0) offsets[e] = at[0];
#pragma unroll
      for (int k = 0; k < kTileMaps; ++k) {
        // the maps are shared out over the workgroups: those of map k take its tiles in turn
        const int groups = min((int)gridDim.x, kTileMaps), sharers = (int)gridDim.x / groups;
        const int turn = (int)blockIdx.x / groups;
        if ((int)blockIdx.x % groups != k % groups || turn >= sharers) continue;
        for (int p = turn * kTileRows[k]; p < tot[i]; p += sharers * kTileRows[k])
          maps.t[k][at[1 + k] + p / kTileRows[k]] = int2{e | min(tot[i] - p, kTileRows[k]) << 16, at[0] + p};
      }
#pragma unroll
      for (int k = 0; k < kTileMaps; ++k) at[1 + k] += (tot[i] + kTileRows[k] - 1) / kTileRows[k];
      at[0] += tot[i];
    }
  }
  __syncthreads();
  for (int b = s0; b < s1; b += 64 * R) {
    if (s1 - s0 > 64 * R) fetch(b);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int s = b + 64 * i + lane;
      const bool in = s < s1;
      const int rank = __popcll(same[i] & ((1ull << lane) - 1));
      const int base = in ? mine[key[i]] : 0;
      wave_sync();
      if (in) {
        order[base + rank] = s;
        if (rank == 0) mine[key[i]] = base + __popcll(same[i]);
      }
      wave_sync();
    }
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
  int32_t* hist = reinterpret_cast<int32_t*>(p + g.hist);
  const int slots = tokens * top_k, nb = g.blocks, per = ((slots + nb - 1) / nb + 63) / 64 * 64;
#define GROUP(W, EMAX, PHASE, blocks)                                                                               \
  hipLaunchKernelGGL((k_group_slots<W, EMAX, PHASE>), dim3(blocks), dim3(64 * W), 0, s, idx, slots, per, E, order, \
                     offsets, counts, hist, maps)
  if (E <= 1024) {
    if (nb == 1) {
      GROUP(4, 1024, 0, 1);
    } else {
      GROUP(4, 1024, 1, nb);
      GROUP(4, 1024, 2, nb);
    }
  } else if (nb == 1) {
    GROUP(4, MOE_MAX_EXPERTS, 0, 1);
  } else {
    GROUP(4, MOE_MAX_EXPERTS, 1, nb);
    GROUP(4, MOE_MAX_EXPERTS, 2, nb);
  }
#undef GROUP
  return hipGetLastError();
}

// out[t] = sum_j gate[t][j] y[t k + j] (j ascending), + residual[t].  VEC: a
// thread takes 16 bytes of columns of one token (8 or 4 of them) and keeps
// the loads of 8 slots in flight (16 of them halved the rate); else one column.
// y is read once: its loads are not kept in the caches.  Bound by reading y:
// 4096 x 16 x 7168 bf16 205 us, 5.7 TB/s; one token 4.8 us, latency.
template <int DT, bool VEC>
__global__ __launch_bounds__(256) void k_combine(const void* __restrict__ y, const float* __restrict__ gate, int top_k,
                                                 unsigned per_row, size_t total, int H, const float* residual,
                                                 float* out) {
  constexpr int N = VEC ? 16 / Elem<DT>::bytes : 1, U = 8;
  const size_t g = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (g >= total) return;
  const size_t t = g / per_row;
  const int h = (int)(g - t * per_row) * N;
  const float* gt = gate + t * top_k;
  const size_t y0 = t * top_k * H + h;
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
  for (int j0 = 0; j0 < top_k; j0 += U) {
    u32x4 c[U];
    float w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(j0 + u, top_k - 1);
      w[u] = gt[j];
      const size_t at = y0 + (size_t)j * H;
      if constexpr (VEC)
        c[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const char*>(y) + at * Elem<DT>::bytes));
      else
        c[u][0] = __float_as_uint(load_f32<DT>(y, at));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j0 + u >= top_k) break;
      float v[N];
      if constexpr (VEC) Chunk<DT>::widen(c[u], v);
      else v[0] = __uint_as_float(c[u][0]);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = fmaf(w[u], v[i], acc[i]);
    }
  }
  const size_t at = t * H + h;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      f32x4 r{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
      if (residual) r += *reinterpret_cast<const f32x4*>(residual + at + i);
      *reinterpret_cast<f32x4*>(out + at + i) = r;
    }
  } else {
    out[at] = residual ? residual[at] + acc[0] : acc[0];
  }
}

template <int DT>
static void combine_dt(const void* y, const float* gate, size_t tokens, int top_k, int H, const float* residual,
                       float* out, hipStream_t s) {
  constexpr int N = 16 / Elem<DT>::bytes;
  auto at16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const bool vec = H % N == 0 && at16(y) && at16(out) && at16(residual);
  const unsigned per_row = vec ? H / N : H;
  const size_t total = tokens * per_row;
  const dim3 grid((unsigned)((total + 255) / 256)), block(256);
  if (vec) hipLaunchKernelGGL((k_combine<DT, true>), grid, block, 0, s, y, gate, top_k, per_row, total, H, residual, out);
  else hipLaunchKernelGGL((k_combine<DT, false>), grid, block, 0, s, y, gate, top_k, per_row, total, H, residual, out);
}

hipError_t launch_combine(const void* y, int dtype, const float* gate, int tokens, int top_k, int H,
                          const float* residual, float* out, hipStream_t s) {
  // a launch holds at most 2^31 threads: long calls go in pieces of whole tokens
  const size_t step = ((size_t)1 << 31) / H;
  for (size_t t0 = 0; t0 < (size_t)tokens; t0 += step) {
    const size_t nt = tokens - t0 < step ? tokens - t0 : step;
    const void* yp = static_cast<const char*>(y) + t0 * top_k * H * (dtype == MOE_DTYPE_F32 ? 4 : 2);
    const float* gp = gate + t0 * top_k;
    const float* rp = residual ? residual + t0 * H : nullptr;
    float* op = out + t0 * H;
    if (dtype == MOE_DTYPE_BF16) combine_dt<MOE_DTYPE_BF16>(yp, gp, nt, top_k, H, rp, op, s);
    else if (dtype == MOE_DTYPE_F16) combine_dt<MOE_DTYPE_F16>(yp, gp, nt, top_k, H, rp, op, s);
    else combine_dt<MOE_DTYPE_F32>(yp, gp, nt, top_k, H, rp, op, s);
  }
  return hipGetLastError();
}

}  // namespace moe
