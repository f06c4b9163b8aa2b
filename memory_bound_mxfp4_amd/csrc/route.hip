// route.hip -- router logits to experts and gates: softmax or sigmoid scores,
// a bias for the selection, groups, top-k, renormalised gates.
//
// One wave per row.  With G groups, group g belongs to L = 64 / G (rounded
// down to a power of two) lanes; lane sub of them holds its experts sub,
// sub + L, ...  (one group: lane l holds l, l + 64, ...).
//
// What decides between two experts is compared as the formula's value in
// fp64: two fp32 scores can tie, or turn round, where the formula does not.
// But fp64 exponentials of all experts are only computed where they enter a
// comparison or a gate: softmax with a bias or without renormalisation (their sum; a short
// form of them in the latter), and groups whose worth is more
// than their best logit.  Otherwise the selection works on an fp32 key per
// expert: the logit itself without a bias (the scores grow with it), the fp32
// score + bias with one.  The k-th largest of the lanes' best keys, T, is no
// better than the k-th best expert (the lanes are disjoint), so only experts
// with keys >= T (with a bias: T less what fp32 may be off) can be among the
// best k: about 20 of 896 at k 16.  They move to one lane each, get their
// exact 64-bit key there, and are ranked against each other.  Ties in a
// logit are cut by index already at T.  More than 64 survivors go the slow way: k rounds
// over all experts, with a bias an exponential of each in every round.  That takes equal
// scores under a bias, a top_k above about 36, or groups that leave fewer lanes than top_k
// (then T is 0).  4096 rows of 896: top 48 255 us, 557 with a bias and sigmoid, top 64 338 us; of
// 1024 in 8 groups, 4 kept, top 32: 192 and 427 us (16384 rows of 896, top 16: 26 us).
//
// A long call of the usual kind is bound by vector instructions (16384 rows of 896 experts,
// sigmoid with a bias, top 16: 26 us, 2.3 TB/s; 706 of them a row, issuing 70% of the time, a
// third for the 896 scores and a quarter for the survivors in fp64), a short one by
// latency (one row of 896: 5.0 us; 4093 rows of 160 in 8 groups by
// their best: 7.3 us).
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

// As dpp_u32, with 0 for a lane that has no source.
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ uint32_t dpp_or_0(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW_MASK, 0xF, false);
}

// A T with at least k lanes holding v >= T: the largest such T, or a smaller one
// with at most k + slack lanes above it; 0 if fewer than k hold more than 0.
// held: how many hold v >= T.  close: start below the bits that all values share, which
// pays for scores with a bias (16384 rows of 896: 27.4 us for 28.8) and not for
// logits (one row: 5.5 us for 5.4).
template <int BITS>
__device__ __forceinline__ uint32_t kth_largest(uint32_t v, int k, int slack, bool close, int& held) {
  static_assert(BITS % 2 == 0, "two bits a round: a round costs a branch and little else");
  uint32_t t = 0;
  int top = BITS - 2;
  held = 64;
  if (close) {
    const int some = __popcll(__ballot(v != 0));
    if (some < k) return 0;
    held = some;
    const uint32_t hi = wave_max_u32(v), differ = hi ^ wave_min_u32(v ? v : hi);
    if (!differ) return hi;
    top = (31 - __clz((int)differ)) & ~1;
    t = top + 2 < 32 ? hi >> (top + 2) << (top + 2) : 0u;
  }
#pragma unroll 1
  for (int b = top; b >= 0; b -= 2) {
    const uint32_t c1 = t | (1u << b), c2 = t | (2u << b), c3 = t | (3u << b);
    const int n1 = __popcll(__ballot(v >= c1)), n2 = __popcll(__ballot(v >= c2)), n3 = __popcll(__ballot(v >= c3));
    const int n = n3 >= k ? n3 : n2 >= k ? n2 : n1;
    t = n3 >= k ? c3 : n2 >= k ? c2 : n1 >= k ? c1 : t;
    held = n >= k ? n : held;
    if (n >= k && n <= k + slack) break;
  }
  return t;
}

// exp(v - top) for v <= top, a term of a softmax's sum: within 2^-29 of itself down to
// e^-100, and that instead of anything smaller (also for -inf), which no sum that holds
// exp(0) can tell.  In fp64, 2^(n + f) with f in -1/2 .. 1/2 and a polynomial of degree 6
// for 2^f (least largest relative error, fitted in fp64); n goes into the exponent.  The
// sum in fp32, of accurate fp32 exponentials, left gates twice as far off (5.4e-8 for
// 2.5e-8 on average) and took up to 8% less (4093 rows of 160: 7.5 us for 7.6; 16384 of 896:
// 28.6 for 31.1; 4096 of 4096: 58.6 for 57.1).
__device__ __forceinline__ double exp_below(float v, double top) {
  constexpr double LOG2E = 1.4426950408889634, MAGIC = 6755399441055744.0;  // 1.5 * 2^52: n in the low bits
  constexpr double C[7] = {1.0000000005541678,  0.6931472057372635,   0.24022646890631455,   0.05550328776970911,
                           0.009618488957365078, 0.001339993121735204, 0.00015345811939447112};
  const double d = fmax((double)v - top, -100.0);
  const double t = fma(d, LOG2E, MAGIC), f = fma(d, LOG2E, MAGIC - t);
  double p = C[6];
#pragma unroll
  for (int k = 5; k >= 0; --k) p = fma(p, f, C[k]);
  const uint64_t bits = __builtin_bit_cast(uint64_t, p);
  const uint32_t hi = (uint32_t)(bits >> 32) + ((uint32_t)__builtin_bit_cast(uint64_t, t) << 20);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | (uint32_t)bits);
}

// GROUPED: L lanes a group; else the row is one group of 64 lanes.
template <int DT, int KPL, bool GROUPED>
__global__ __launch_bounds__(256) void k_route(const void* __restrict__ logits, size_t row_stride, int rows,
                                               const float* __restrict__ bias, moe_route_params p, int lanes,
                                               int32_t* __restrict__ idx_out, float* __restrict__ gate_out) {
  __shared__ float2 list_lb[4][65];  // a survivor's logit and bias
  __shared__ int list_e[4][65];
  __shared__ __attribute__((aligned(16))) uint64_t list_k[4][66];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int row_i = blockIdx.x * 4 + wv;
  if (row_i >= rows) return;
  const size_t row = row_i, base = row * row_stride;
  const int L = GROUPED ? lanes : 64, size = GROUPED ? p.num_experts / p.groups : p.num_experts;
  const int grp = GROUPED ? lane / L : 0, sub = GROUPED ? lane & (L - 1) : lane;
  const int e0 = grp * size;
  int mine = !GROUPED || grp < p.groups ? size : 0;  // experts of this lane: e0 + sub + L i, sub + L i < mine
  const bool softmax = p.score == MOE_SCORE_SOFTMAX;
  const float LOWEST = -__builtin_inff();

  // the logit of a candidate, else -inf
  auto logit = [&](int at) {
    const float v = load_f32<DT>(logits, base + e0 + at), b = bias ? bias[e0 + at] : 0.0f;
    return v > LOWEST && b > LOWEST ? fminf(v, __FLT_MAX__) : LOWEST;  // both false for NaN
  };
  // c: first the logits, then the keys; -inf or NaN: no candidate
  float l[KPL], b[KPL], c[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int at = sub + L * i;
    l[i] = LOWEST;
    if (!GROUPED && 64 * (i + 1) <= size) l[i] = load_f32<DT>(logits, base + at);
    else if (at < mine) l[i] = load_f32<DT>(logits, base + e0 + at);
  }
  if (bias) {
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int at = sub + L * i;
      b[i] = LOWEST;
      if (!GROUPED && 64 * (i + 1) <= size) b[i] = bias[at];
      else if (at < mine) b[i] = bias[e0 + at];
    }
  }
  if (!bias || softmax) {
#pragma unroll
    for (int i = 0; i < KPL; ++i) l[i] = l[i] > LOWEST && (!bias || b[i] > LOWEST) ? fminf(l[i], __FLT_MAX__) : LOWEST;
  }
  float best = LOWEST, top = 0.0f;
  double z = 1.0;
  // a group's worth is its best score alone: then its best logit decides, and no score is needed
  const bool by_logit = GROUPED && !bias && p.group_top == 1;
  double ex[KPL <= 8 ? KPL : 1];  // softmax: the exponentials, where all of them are needed in fp64
  if (softmax) {
#pragma unroll
    for (int i = 0; i < KPL; ++i) best = fmaxf(best, l[i]);
    const uint32_t m = wave_max_u32(best > LOWEST ? order_key(best) : 0u);
    top = m ? order_value(m) : 0.0f;
    if (bias || (GROUPED && !by_logit)) {
      double sum = 0.0;
      if constexpr (KPL <= 8) {
#pragma unroll
        for (int i = 0; i < KPL; ++i) {
          ex[i] = l[i] > LOWEST ? exp((double)l[i] - (double)top) : 0.0;
          sum += ex[i];
        }
      } else {  // one after the other: unrolled, the exponentials of 16 and more take all registers
#pragma unroll 1
        for (int at = sub; at < mine; at += L) {
          const float v = logit(at);
          if (v > LOWEST) sum += exp((double)v - (double)top);
        }
      }
      z = sum_lanes_f64<64>(sum);
    } else if (!p.renorm) {
      double part[4] = {};
#pragma unroll
      for (int i = 0; i < KPL; ++i) part[i % 4] += exp_below(l[i], (double)top);
      z = sum_lanes_f64<64>((part[0] + part[1]) + (part[2] + part[3]));
    }
    if (z == 0.0) z = 1.0;
  }
  auto score = [&](float v) {
    v = fminf(v, __FLT_MAX__);
    return softmax ? exp((double)v - (double)top) / z : 1.0 / (1.0 + exp(-(double)v));
  };
  if (bias) {
    const float rz = (float)(1.0 / z);
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const float s = softmax ? __expf(l[i] - top) * rz : __builtin_amdgcn_rcpf(1.0f + __expf(-l[i]));
      c[i] = l[i] > LOWEST ? s + b[i] : LOWEST;
    }
  } else {
#pragma unroll
    for (int i = 0; i < KPL; ++i) c[i] = l[i];
  }
  if (GROUPED) {
    // the two best of each group, first in a lane, then over its lanes
    const double NONE = -__builtin_inf();
    double b1 = NONE, b2 = NONE;
    auto take = [&](double t) {
      b2 = fmax(b2, fmin(b1, t));
      b1 = fmax(b1, t);
    };
    if (by_logit) {
#pragma unroll
      for (int i = 0; i < KPL; ++i) b1 = fmax(b1, (double)c[i]);
    } else if constexpr (KPL <= 8) {
      const double rz = 1.0 / z;
#pragma unroll
      for (int i = 0; i < KPL; ++i)
        take(c[i] >= -__FLT_MAX__ ? (softmax ? ex[i] * rz : score(l[i])) + (bias ? (double)b[i] : 0.0) : NONE);
    } else {
#pragma unroll 1
      for (int at = sub; at < mine; at += L) {
        const float v = logit(at);
        if (v > LOWEST) take(score(v) + (bias ? (double)bias[e0 + at] : 0.0));
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
    for (int g0 = 0; g0 < p.groups; g0 += 4) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int g = g0 + u;
        const uint64_t o = readlane64(w, min(g * L, 63));
        before += g < p.groups && (o > w || (o == w && g < grp));
      }
    }
    if (!any || before >= p.top_groups) {
      mine = 0;
#pragma unroll
      for (int i = 0; i < KPL; ++i) c[i] = LOWEST;
    }
  }
  best = LOWEST;
#pragma unroll
  for (int i = 0; i < KPL; ++i) best = fmaxf(best, c[i]);
  const uint32_t best_key = best > LOWEST ? order_key(best) : 0u;
  int held, last_tied = MOE_MAX_EXPERTS;  // of the experts with key T, those up to this index survive
  const uint32_t cut_key = kth_largest<32>(best_key, p.top_k, 4, bias != nullptr, held);
  // below 2^23 in this order lie the NaN and -inf: fewer than k candidates
  float cut = cut_key < 0x00800000u ? -__FLT_MAX__ : order_value(cut_key);
  if (bias) {
    // fp32 score: under 2^-21 off (exponential, reciprocal, a score is at most
    // 1); the sum: half a step.  Twice that on both sides of T.
    if (cut <= __FLT_MAX__) cut = fmaxf(cut - (0x1p-19f + fabsf(cut) * 0x1p-22f), -__FLT_MAX__);
  } else if (held > p.top_k + 4 && cut_key) {
    // a tie at T: only the lowest indices of those lanes that hold it can come in
    uint32_t low = 0;
#pragma unroll
    for (int i = KPL - 1; i >= 0; --i)
      if (c[i] == cut) low = 0xFFFu - (uint32_t)(e0 + sub + L * i);
    const int above = __popcll(__ballot(best_key > cut_key));
    int unused;
    last_tied = 0xFFF - (int)kth_largest<12>(best_key == cut_key ? low : 0u, p.top_k - above, 0, false, unused);
  }
  // The survivors of each lane one after another.
  auto survives = [&](int i) {
    return c[i] >= cut && (last_tied == MOE_MAX_EXPERTS || c[i] > cut || e0 + sub + L * i <= last_tied);
  };
  uint32_t mine_in = 0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) mine_in += survives(i) ? 1u : 0u;
  uint32_t at = mine_in;
  at += dpp_or_0<0x111>(at);       // row_shr:1
  at += dpp_or_0<0x112>(at);       // row_shr:2
  at += dpp_or_0<0x114>(at);       // row_shr:4
  at += dpp_or_0<0x118>(at);       // row_shr:8
  at += dpp_or_0<0x142, 0xA>(at);  // row_bcast:15 into rows 1, 3
  at += dpp_or_0<0x143, 0xC>(at);  // row_bcast:31 into rows 2, 3
  const int n = __builtin_amdgcn_readlane((int)at, 63);
  at -= mine_in;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    if (!survives(i)) continue;
    const int place = min((int)at, 64);
    list_e[wv][place] = e0 + sub + L * i;
    list_lb[wv][place] = float2{l[i], bias ? b[i] : 0.0f};
    ++at;
  }
  wave_sync();
  int e = -1, place = lane;  // without an expert: places from n on stay empty
  double s = 0.0;
  if (n <= 64) {
    // Keys with the index behind them, so that no two are alike: the logit's 32
    // bits, or the first 52 of the fp64 score + bias.
    uint64_t exact = 0, k64 = 0;
    if (lane < n) {
      e = list_e[wv][lane];
      const float2 lb = list_lb[wv][lane];
      s = score(lb.x);
      exact = bias ? order64(s + (double)lb.y) : (uint64_t)order_key(lb.x);
      k64 = bias ? (exact & ~0xFFFull) | (uint64_t)(0xFFF - e) : (exact << 32) | (uint64_t)(0xFFF - e);
    }
    list_k[wv][lane] = k64;
    wave_sync();
    int ahead = 0;
    for (int j = 0; j < n; j += 2) {
      typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
      const u64x2 o = *reinterpret_cast<const u64x2*>(&list_k[wv][j]);
      ahead += (o[0] > k64) + (o[1] > k64);
    }
    if (bias) {
      // two neighbours with the same 52 bits: all of them, then the index, decide
      wave_sync();
      if (lane < n) list_k[wv][ahead] = k64;
      wave_sync();
      const bool close = lane < n && ahead + 1 < n && (list_k[wv][ahead + 1] >> 12) == (k64 >> 12);
      if (__ballot(close)) {
        ahead = 0;
        for (int j = 0; j < n; ++j) {
          const uint64_t o = readlane64(exact, j);
          const int oe = __builtin_amdgcn_readlane(e, j);
          ahead += o > exact || (o == exact && oe < e);
        }
      }
    }
    if (lane < n) place = ahead;
  } else {
    // lane j takes the best expert after the one of place j - 1
    uint64_t last_k = ~0ull;
    int last_e = -1;
#pragma unroll 1
    for (int j = 0; j < p.top_k; ++j) {
      uint64_t bk = 0;
      int be = MOE_MAX_EXPERTS;
#pragma unroll 1
      for (int at = sub; at < mine; at += L) {
        const int x = e0 + at;
        const float v = logit(at);
        if (!(v > LOWEST)) continue;
        const uint64_t k = bias ? order64(score(v) + (double)bias[x]) : (uint64_t)order_key(v);
        if ((k < last_k || (k == last_k && x > last_e)) && k > bk) {
          bk = k;
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
    if (e >= 0) s = score(load_f32<DT>(logits, base + e));
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
#define ROUTE(KPL)                                                                                                   \
  if (p.groups > 1)                                                                                                  \
    hipLaunchKernelGGL((k_route<DT, KPL, true>), grid, block, 0, s, logits, row_stride, rows, bias, p, L, idx, gate); \
  else                                                                                                               \
    hipLaunchKernelGGL((k_route<DT, KPL, false>), grid, block, 0, s, logits, row_stride, rows, bias, p, L, idx, gate)
  if (kpl <= 1) {
    ROUTE(1);
  } else if (kpl <= 2) {
    ROUTE(2);
  } else if (kpl <= 4) {
    ROUTE(4);
  } else if (kpl <= 8) {
    ROUTE(8);
  } else if (kpl <= 16) {
    ROUTE(16);
  } else if (kpl <= 32) {
    ROUTE(32);
  } else if (kpl <= 64) {
    ROUTE(64);
  } else {  // many groups leave a lane up to 124 experts
    hipLaunchKernelGGL((k_route<DT, 128, true>), grid, block, 0, s, logits, row_stride, rows, bias, p, L, idx, gate);
  }
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
