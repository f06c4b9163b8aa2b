// route.hip -- router logits to experts and gates: softmax or sigmoid scores,
// a bias for the selection, groups, top-k, renormalised gates.
//
// One wave per row.  With G groups, group g belongs to L = 64 / G (rounded
// down to a power of two) lanes; lane sub of them holds its experts sub,
// sub + L, ...  (one group: lane l holds l, l + 64, ...).
//
// What decides between two experts is compared as the formula's value in
// fp64: two fp32 scores can tie, or turn round, where the formula does not.
// But fp64 exponentials of all experts are only computed where a sum of all
// of them enters the comparison (softmax with a bias) or every expert may
// count for its group.  Otherwise the selection works on a 32-bit key per
// expert: the logit itself without a bias (the scores grow with it), the fp32
// score + bias with one.  The k-th largest of the lanes' best keys, T, is no
// better than the k-th best expert (the lanes are disjoint), so only experts
// with keys >= T (with a bias: T less what fp32 may be off) can be among the
// best k: about 20 of 896 at k 16.  They move to one lane each, get their
// exact 64-bit key there, and are ranked against each other.  Ties in a
// logit are cut by index already at T.  More than 64 survivors (equal scores
// under a bias, or a large k) go the slow way: k rounds over all experts.
#include "i8_common.h"
#include "moe_device.h"

namespace moe {

__device__ __forceinline__ uint64_t order64(double c) {
  const uint64_t u = __builtin_bit_cast(uint64_t, c == 0.0 ? 0.0 : c);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

__device__ __forceinline__ uint64_t readlane64(uint64_t v, int l) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), l);
  return ((uint64_t)hi << 32) | lo;
}

// The largest T with at least k lanes holding v >= T (0 if fewer than k hold
// more than 0), and how many hold v >= T.
template <int BITS>
__device__ __forceinline__ uint32_t kth_largest(uint32_t v, int k, int& held) {
  uint32_t t = 0;
  held = 64;
#pragma unroll 1
  for (int b = BITS - 1; b >= 0; --b) {
    const uint32_t c = t | (1u << b);
    const int n = __popcll(__ballot(v >= c));
    if (n >= k) {
      t = c;
      held = n;
      if (n == k) break;  // T may stay coarse: the same k lanes are above it
    }
  }
  return t;
}

template <int DT, int KPL>
__global__ __launch_bounds__(256) void k_route(const void* __restrict__ logits, size_t row_stride, int rows,
                                               const float* __restrict__ bias, moe_route_params p, int L,
                                               int32_t* __restrict__ idx_out, float* __restrict__ gate_out) {
  __shared__ uint32_t list_e[4][64];
  __shared__ float list_l[4][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int row_i = blockIdx.x * 4 + wv;
  if (row_i >= rows) return;
  const size_t row = row_i, base = row * row_stride;
  const int size = p.num_experts / p.groups, grp = lane / L, sub = lane & (L - 1);
  const int e0 = grp * size;
  int mine = grp < p.groups ? size : 0;  // experts of this lane: e0 + sub + L i, sub + L i < mine
  const bool softmax = p.score == MOE_SCORE_SOFTMAX;
  const float LOWEST = -__builtin_inff();

  // the logit of a candidate, else -inf
  auto logit = [&](int at) {
    const float v = load_f32<DT>(logits, base + e0 + at), b = bias ? bias[e0 + at] : 0.0f;
    return v > LOWEST && b > LOWEST ? fminf(v, __FLT_MAX__) : LOWEST;  // both false for NaN
  };
  uint32_t key[KPL];
  float l[KPL];
  uint32_t best = 0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) l[i] = sub + L * i < mine ? load_f32<DT>(logits, base + e0 + sub + L * i) : LOWEST;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const float b = bias && sub + L * i < mine ? bias[e0 + sub + L * i] : 0.0f;
    l[i] = l[i] > LOWEST && b > LOWEST ? fminf(l[i], __FLT_MAX__) : LOWEST;  // both false for NaN
    key[i] = l[i] > LOWEST ? order_key(l[i]) : 0u;
    best = max(best, key[i]);
  }
  float top = 0.0f;
  double z = 1.0;
  if (softmax) {
    const uint32_t m = wave_max_u32(best);
    top = m ? order_value(m) : 0.0f;
    if (bias || p.groups > 1) {
      double sum = 0.0;
#pragma unroll 1
      for (int at = sub; at < mine; at += L) {
        const float v = logit(at);
        if (v > LOWEST) sum += exp((double)v - (double)top);
      }
      z = sum_lanes_f64<64>(sum);
    } else if (!p.renorm) {
      float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // chains of at most KPL / 4 additions
#pragma unroll
      for (int i = 0; i < KPL; ++i)
        if (l[i] > LOWEST) s4[i & 3] += expf(l[i] - top);
      z = (double)sum_lanes<64>((s4[0] + s4[1]) + (s4[2] + s4[3]));
    }
    if (z == 0.0) z = 1.0;
  }
  auto score = [&](float v) { return softmax ? exp((double)v - (double)top) / z : 1.0 / (1.0 + exp(-(double)v)); };

  if (p.groups > 1) {
    // the two best of each group, first in a lane, then over its lanes
    const double NONE = -__builtin_inf();
    double b1 = NONE, b2 = NONE;
#pragma unroll 1
    for (int at = sub; at < mine; at += L) {
      const float v = logit(at);
      if (v > LOWEST) {
        const double c = score(v) + (bias ? (double)bias[e0 + at] : 0.0);
        b2 = fmax(b2, fmin(b1, c));
        b1 = fmax(b1, c);
      }
    }
    for (int m = L / 2; m >= 1; m >>= 1) {
      const double o1 = __shfl_xor(b1, m, WAVE), o2 = __shfl_xor(b2, m, WAVE);
      b2 = fmax(fmin(b1, o1), fmax(b2, o2));
      b1 = fmax(b1, o1);
    }
    const bool any = b1 > NONE;
    const double worth = !any ? NONE : p.group_top == 2 && b2 > NONE ? b1 + b2 : b1;
    const uint64_t w = order64(worth);
    int before = 0;
    for (int g = 0; g < p.groups; ++g) {
      const uint64_t o = readlane64(w, g * L);
      before += o > w || (o == w && g < grp);
    }
    if (!any || before >= p.top_groups) {
      mine = 0;
#pragma unroll
      for (int i = 0; i < KPL; ++i) key[i] = 0u;
    }
  }
  uint32_t cut_key, cut_low = 0;  // survivors: key > cut_key, or equal and ~index >= cut_low
  if (bias) {
    const float rz = (float)(1.0 / z);
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const float s = softmax ? __expf(l[i] - top) * rz : __builtin_amdgcn_rcpf(1.0f + __expf(-l[i]));
      if (key[i]) key[i] = order_key(s + bias[e0 + sub + L * i]);
    }
  }
  best = 0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) best = max(best, key[i]);
  int held;
  cut_key = kth_largest<32>(best, p.top_k, held);
  if (bias) {
    // fp32 score: under 2^-21 off (exponential, reciprocal, a score is at most
    // 1); the sum: half a step.  Twice that on both sides of T.
    const float t = order_value(cut_key);
    if (cut_key && fabsf(t) <= __FLT_MAX__) cut_key = order_key(t - (0x1p-19f + fabsf(t) * 0x1p-22f));
  } else if (held > p.top_k && cut_key) {
    // a tie at T: only the lowest indices of those lanes that hold it can come in
    uint32_t low = 0;
#pragma unroll
    for (int i = KPL - 1; i >= 0; --i)
      if (key[i] == cut_key) low = 0xFFFu - (uint32_t)(e0 + sub + L * i);
    const int above = __popcll(__ballot(best > cut_key));
    int unused;
    cut_low = kth_largest<12>(best == cut_key ? low : 0u, p.top_k - above, unused);
  }
  cut_key = max(cut_key, 1u);  // key 0: no candidate
  int n = 0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const uint32_t e = (uint32_t)(e0 + sub + L * i);
    const bool in = key[i] > cut_key || (key[i] == cut_key && 0xFFFu - e >= cut_low);
    const uint64_t m = __ballot(in);
    const int at = n + __popcll(m & ((1ull << lane) - 1));
    if (in && at < 64) {
      list_e[wv][at] = e;
      if (!bias) list_l[wv][at] = order_value(key[i]);
    }
    n += __popcll(m);
  }
  __builtin_amdgcn_wave_barrier();
  int e = -1, place = 64;
  double s = 0.0;
  if (n <= 64) {
    uint64_t k64 = 0;
    if (lane < n) {
      e = (int)list_e[wv][lane];
      const float v = bias ? fminf(load_f32<DT>(logits, base + e), __FLT_MAX__) : list_l[wv][lane];
      s = score(v);
      k64 = bias ? order64(s + (double)bias[e]) : (uint64_t)order_key(v);
    }
    place = 0;
    for (int j = 0; j < n; ++j) {
      const uint64_t o = readlane64(k64, j);
      const int oe = __builtin_amdgcn_readlane(e, j);
      place += o > k64 || (o == k64 && oe < e);
    }
    if (lane >= n) place = lane;  // fewer candidates than places: these stay empty
  } else {
    // lane j takes the best expert after the one of place j - 1
    uint64_t last_k = ~0ull;
    int last_e = -1;
    place = lane;
#pragma unroll 1
    for (int j = 0; j < p.top_k; ++j) {
      uint64_t bk = 0;
      int be = MOE_MAX_EXPERTS;
#pragma unroll 1
      for (int at = sub; at < mine; at += L) {
        const int x = e0 + at;
        const float v = logit(at);
        if (!(v > LOWEST)) continue;
        const uint64_t c = bias ? order64(score(v) + (double)bias[x]) : (uint64_t)order_key(v);
        if ((c < last_k || (c == last_k && x > last_e)) && c > bk) {
          bk = c;
          be = x;
        }
      }
#pragma unroll
      for (int m = 32; m >= 1; m >>= 1) {
        const uint64_t o = shfl_xor_u64(bk, m);
        const int oe = __shfl_xor(be, m, WAVE);
        if (o > bk || (o == bk && oe < be)) {
          bk = o;
          be = oe;
        }
      }
      last_k = bk;
      last_e = be;
      if (lane == j) e = be;
    }
    if (e >= 0) s = score(fminf(load_f32<DT>(logits, base + e), __FLT_MAX__));
  }
  if (place >= p.top_k) s = 0.0;
  if (p.renorm) {
    const double sum = sum_lanes_f64<64>(s);
    s = sum > 0.0 ? s / sum : 0.0;
  }
  if (place < p.top_k) {
    idx_out[row * p.top_k + place] = e;
    gate_out[row * p.top_k + place] = (float)(s * (double)p.scale);
  }
}

template <int DT>
static void route_dt(const void* logits, size_t row_stride, int rows, const float* bias, const moe_route_params& p,
                     int32_t* idx, float* gate, hipStream_t s) {
  int L = 64;
  while (L * p.groups > 64) L >>= 1;
  const int kpl = (p.num_experts / p.groups + L - 1) / L;
  const dim3 grid((rows + 3) / 4), block(256);
#define ROUTE(KPL) \
  hipLaunchKernelGGL((k_route<DT, KPL>), grid, block, 0, s, logits, row_stride, rows, bias, p, L, idx, gate)
  if (kpl <= 1) ROUTE(1);
  else if (kpl <= 2) ROUTE(2);
  else if (kpl <= 4) ROUTE(4);
  else if (kpl <= 8) ROUTE(8);
  else if (kpl <= 16) ROUTE(16);
  else if (kpl <= 32) ROUTE(32);
  else if (kpl <= 64) ROUTE(64);
  else ROUTE(128);
#undef ROUTE
}

hipError_t launch_route(const void* logits, int dtype, size_t row_stride, int rows, const float* bias,
                        const moe_route_params& p, int32_t* idx, float* gate, hipStream_t s) {
  if (dtype == MOE_DTYPE_BF16) route_dt<MOE_DTYPE_BF16>(logits, row_stride, rows, bias, p, idx, gate, s);
  else if (dtype == MOE_DTYPE_F16) route_dt<MOE_DTYPE_F16>(logits, row_stride, rows, bias, p, idx, gate, s);
  else route_dt<MOE_DTYPE_F32>(logits, row_stride, rows, bias, p, idx, gate, s);
  return hipGetLastError();
}

}  // namespace moe
