// route.hip -- router logits to experts and gates: softmax or sigmoid scores,
// a bias for the selection, groups, top-k, renormalised gates.
//
// One wave per row; lane l holds experts l, l + 64, ...  Whatever decides
// between two experts is computed in fp64: a comparison of two fp32 scores
// would tie, or turn round, where the formula does not.
#include "i8_common.h"

namespace moe {

__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = fmax(v, __shfl_xor(v, m, WAVE));
  return v;
}
__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, WAVE));
  return v;
}
__device__ __forceinline__ int wave_min_i32(int v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = min(v, __shfl_xor(v, m, WAVE));
  return v;
}

template <int DT, int KPL>
__global__ __launch_bounds__(64) void k_route(const void* __restrict__ logits, size_t row_stride,
                                              const float* __restrict__ bias, moe_route_params p,
                                              int32_t* __restrict__ idx_out, float* __restrict__ gate_out) {
  const size_t row = blockIdx.x;
  const int lane = threadIdx.x, E = p.num_experts;
  const double NONE = -__builtin_inf();
  float l[KPL];
  uint64_t cand = 0;
  float top = -__FLT_MAX__;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int e = lane + 64 * i;
    l[i] = 0.0f;
    if (e < E) {
      const float v = load_f32<DT>(logits, row * row_stride + e), b = bias ? bias[e] : 0.0f;
      l[i] = fminf(v, __FLT_MAX__);
      if (v > -__builtin_inff() && b > -__builtin_inff()) {  // false for NaN too
        cand |= 1ull << i;
        top = fmaxf(top, l[i]);
      }
    }
  }
  top = wave_max_f32(top);
  const bool softmax = p.score == MOE_SCORE_SOFTMAX;
  double c[KPL], z = 0.0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    c[i] = 0.0;
    if ((cand >> i) & 1) c[i] = softmax ? exp((double)l[i] - (double)top) : 1.0 / (1.0 + exp(-(double)l[i]));
    z += c[i];
  }
  z = sum_lanes_f64<64>(z);
  if (!softmax || z == 0.0) z = 1.0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int e = lane + 64 * i;
    c[i] = ((cand >> i) & 1) ? c[i] / z + (bias ? (double)bias[e] : 0.0) : NONE;
  }
  if (p.groups > 1) {
    const int size = E / p.groups;
    double worth = NONE;  // lane g: the worth of group g
    for (int g = 0; g < p.groups; ++g) {
      double w = 0.0;
      int gone = -1;
      bool any = false;
      for (int j = 0; j < p.group_top; ++j) {
        double best = NONE;
        int at = E;
#pragma unroll
        for (int i = 0; i < KPL; ++i) {
          const int e = lane + 64 * i;
          if (e >= g * size && e < (g + 1) * size && e != gone && c[i] > best) {
            best = c[i];
            at = e;
          }
        }
        const double m = wave_max_f64(best);
        gone = wave_min_i32(best == m ? at : E);
        if (m > NONE) {
          w += m;
          any = true;
        }
      }
      if (lane == g && any) worth = w;
    }
    uint64_t kept = 0;
    for (int j = 0; j < p.top_groups; ++j) {
      const double m = wave_max_f64(worth);
      if (!(m > NONE)) break;
      const int g = wave_min_i32(worth == m ? lane : 64);
      kept |= 1ull << g;
      if (lane == g) worth = NONE;
    }
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((kept >> (e / size)) & 1)) {
        c[i] = NONE;
        cand &= ~(1ull << i);
      }
    }
  }
  if (!bias) {
#pragma unroll
    for (int i = 0; i < KPL; ++i) c[i] = ((cand >> i) & 1) ? (double)l[i] : NONE;
  }
  int mine = -1;
  for (int j = 0; j < p.top_k; ++j) {
    double best = NONE;
    int at = E;
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if (c[i] > best) {
        best = c[i];
        at = lane + 64 * i;
      }
    const double m = wave_max_f64(best);
    if (!(m > NONE)) break;
    const int e = wave_min_i32(best == m ? at : E);
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if (lane + 64 * i == e) c[i] = NONE;
    if (lane == j) mine = e;
  }
  double s = 0.0;
  if (mine >= 0) {
    const double v = (double)fminf(load_f32<DT>(logits, row * row_stride + mine), __FLT_MAX__);
    s = softmax ? exp(v - (double)top) / z : 1.0 / (1.0 + exp(-v));
  }
  if (p.renorm) {
    const double sum = sum_lanes_f64<64>(s);
    s = sum > 0.0 ? s / sum : 0.0;
  }
  if (lane < p.top_k) {
    idx_out[row * p.top_k + lane] = mine;
    gate_out[row * p.top_k + lane] = (float)(s * (double)p.scale);
  }
}

template <int DT>
static void route_dt(const void* logits, size_t row_stride, int rows, const float* bias, const moe_route_params& p,
                     int32_t* idx, float* gate, hipStream_t s) {
  const dim3 grid(rows), block(64);
  const int kpl = (p.num_experts + 63) / 64;
  if (kpl <= 1) hipLaunchKernelGGL((k_route<DT, 1>), grid, block, 0, s, logits, row_stride, bias, p, idx, gate);
  else if (kpl <= 2) hipLaunchKernelGGL((k_route<DT, 2>), grid, block, 0, s, logits, row_stride, bias, p, idx, gate);
  else if (kpl <= 4) hipLaunchKernelGGL((k_route<DT, 4>), grid, block, 0, s, logits, row_stride, bias, p, idx, gate);
  else if (kpl <= 8) hipLaunchKernelGGL((k_route<DT, 8>), grid, block, 0, s, logits, row_stride, bias, p, idx, gate);
  else if (kpl <= 16) hipLaunchKernelGGL((k_route<DT, 16>), grid, block, 0, s, logits, row_stride, bias, p, idx, gate);
  else if (kpl <= 32) hipLaunchKernelGGL((k_route<DT, 32>), grid, block, 0, s, logits, row_stride, bias, p, idx, gate);
  else hipLaunchKernelGGL((k_route<DT, 64>), grid, block, 0, s, logits, row_stride, bias, p, idx, gate);
}

hipError_t launch_route(const void* logits, int dtype, size_t row_stride, int rows, const float* bias,
                        const moe_route_params& p, int32_t* idx, float* gate, hipStream_t s) {
  if (dtype == MOE_DTYPE_BF16) route_dt<MOE_DTYPE_BF16>(logits, row_stride, rows, bias, p, idx, gate, s);
  else if (dtype == MOE_DTYPE_F16) route_dt<MOE_DTYPE_F16>(logits, row_stride, rows, bias, p, idx, gate, s);
  else route_dt<MOE_DTYPE_F32>(logits, row_stride, rows, bias, p, idx, gate, s);
  return hipGetLastError();
}

}  // namespace moe
