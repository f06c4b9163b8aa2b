// norm_q.hip -- the residual's addition, the root-mean-square norm and its
// output as 8-bit codes with scales, a row read once.
//
//   g = h + t (fp32, stored),  v = g / sqrt(mean(g^2) + eps) * gain,
//   codes and scales of v as the quantisers have them
//
// The sum of squares, v and the quotients v / scale are computed in fp64 (a 24 x 24 bit
// product fits without rounding), so the codes are those of the formula, but for v within
// some 2^-50 of the middle between two.  The vector units have the time: a row waits for memory
// (16384 rows of 7168, t of bf16, e4m3 codes: 240 us, 5.4 TB/s; a large copy has 5.0; one row 5.2, latency).
#include <float.h>

#include "f8_common.h"

namespace moe {

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, WAVE);
  return v;
}
template <int LANES>
__device__ __forceinline__ double lanes_max64(double v) {
#pragma unroll
  for (int d = LANES / 2; d >= 1; d >>= 1) v = fmax(v, __shfl_xor(v, d, WAVE));
  return v;
}

// A scale and what 8-bit codes of values a * inv are computed with.
struct NormScale {
  float stored;
  double mul;  // the quotient is a * mul
  bool zero;
};
// amax: the largest |a| (infinity where a is not finite); inv: NaN for a row that is not finite.
__device__ __forceinline__ NormScale norm_scale(double amax, double inv, double most) {
  NormScale r;
  const float s = (float)(amax * inv / most);
  const bool bad = !(s <= FLT_MAX);
  r.stored = bad ? __uint_as_float(0x7FC00000u) : s;
  r.zero = bad || s == 0.0f;
  r.mul = r.zero ? 0.0 : inv / (double)s;
  return r;
}

// A quotient to the fp32 number that converts to its nearest e4m3 value: rounded to fp32
// first, it could only go wrong where that lands on a middle.
__device__ __forceinline__ float f8_quotient(double q) {
  float t = f8_clamp((float)q);
  if (f8_near<0>(t)) {
    const float m = f8_middle(t);
    t = f8_side(t, m, fabs(q) - (double)m);
  }
  return t;
}

// T threads a row, each with chunks of 8 elements tid, tid + T, ...; NC > 0: at most NC of
// them, kept in registers; NC 0: any number, read again from memory (h_out, which the same
// thread wrote) for each of the later passes.
template <int DT, bool F8, bool VEC, int T, int NC>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_norm_q(NormArgs a) {
  constexpr int B = T < 256 ? 256 : T, W = T / 64, R = NC ? NC : 1;
  __shared__ double part[W];
  const int tid = threadIdx.x % T, lane = threadIdx.x & 63, wv = tid >> 6;
  const size_t row = a.row0 + (size_t)blockIdx.x * (B / T) + threadIdx.x / T;
  if (B != T && row >= (size_t)a.rows) return;
  const int H = a.hidden, blocks = (H + kBlock - 1) / kBlock, chunks = blocks * kLanes;
  const float* hrow = a.h + row * a.h_stride;
  const char* trow = static_cast<const char*>(a.t) + row * a.t_stride * Elem<DT>::bytes;
  float* orow = a.h_out + row * H;
  float g[R][8];

  // A chunk of h and t; then their sum, stored.  (Apart: h_out may be h, so no load moves over a store.)
  auto fetch = [&](int c, float* v, float* u) {
    load8<MOE_DTYPE_F32, VEC>(hrow, c, H, v);
    if (a.t) load8<DT, VEC>(trow, c, H, u);
  };
  auto sum = [&](int c, float* v, const float* u) {
    if (!a.t) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += u[i];
    if constexpr (VEC) {
      if (8 * c >= H) return;
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        *reinterpret_cast<f32x4*>(orow + 8 * c + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (element<VEC>(c, i) < H) orow[element<VEC>(c, i)] = v[i];
    }
  };
  auto again = [&](int c, float* v) { load8<MOE_DTYPE_F32, VEC>(a.t ? orow : hrow, c, H, v); };  // in a later pass
  auto squares = [&](const float* v, double s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fma((double)v[i], (double)v[i], s);
    return s;
  };
  auto row_sum = [&](double v) {
    v = wave_sum64(v);
    if constexpr (W > 1) {
      if (lane == 0) part[wv] = v;
      __syncthreads();
      v = part[0];
#pragma unroll
      for (int i = 1; i < W; ++i) v += part[i];
    }
    return v;
  };

  double ss = 0.0;
  if constexpr (NC > 0) {
    float u[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) fetch(tid + T * i, g[i], u[i]);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      sum(tid + T * i, g[i], u[i]);
      ss = squares(g[i], ss);
    }
  } else {
    for (int c = tid; c < chunks; c += T) {
      float u[8];
      fetch(c, g[0], u);
      sum(c, g[0], u);
      ss = squares(g[0], ss);
    }
  }
  ss = row_sum(ss);
  const double inv = ss <= DBL_MAX ? 1.0 / sqrt(ss / H + (double)a.eps) : __longlong_as_double(0x7FF8000000000000ll);

  // g * gain of a chunk, and the largest of them
  auto gained = [&](int c, const float* v, double* p) {
    float w[8];
    if (a.gain) {
      load8<MOE_DTYPE_F32, VEC>(a.gain, c, H, w);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    }
    uint32_t most = 0;
    double m = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = (double)v[i] * (double)w[i];
      m = fmax(m, fabs(p[i]));
      most = max(most, abs_bits(w[i]));
    }
    return most >= 0x7F800000u ? __longlong_as_double(0x7FF0000000000000ll) : m;
  };
  auto put_out = [&](int c, const double* p) {  // the normalised chunk in bf16
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)(p[i] * inv);
    uint16_t* o = a.out + row * H;
    if constexpr (VEC) {
      if (8 * c >= H) return;
      u32x4 d;
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = pack2<MOE_DTYPE_BF16>(v[2 * i], v[2 * i + 1]);
      reinterpret_cast<u32x4*>(o)[c] = d;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (element<VEC>(c, i) < H) o[element<VEC>(c, i)] = f32_to_bf16(v[i]);
    }
  };

  if constexpr (F8) {
    auto block = [&](int c, const float* v) {
      double p[8];
      const double m = lanes_max64<kLanes>(gained(c, v, p));
      const NormScale s = norm_scale(m, inv, 448.0);
      if (tid % kLanes == 0) a.scale[(size_t)(c / kLanes) * a.rows + row] = s.stored;
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = f8_quotient(p[i] * s.mul);
      store8_codes<VEC>(static_cast<uint8_t*>(a.q) + row * H, c, H, s.zero ? u32x2{0u, 0u} : f8_pack(t));
      if (a.out) put_out(c, p);
    };
    // a block's 16 lanes take the same turn: T is a multiple of them
    if constexpr (NC > 0) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (tid + T * i < chunks) block(tid + T * i, g[i]);
    } else {
      for (int c = tid; c < chunks; c += T) {
        again(c, g[0]);
        block(c, g[0]);
      }
    }
  } else {
    double m = 0.0, p[8];
    if constexpr (NC > 0) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (tid + T * i < chunks) m = fmax(m, gained(tid + T * i, g[i], p));
    } else {
      for (int c = tid; c < chunks; c += T) {
        again(c, g[0]);
        m = fmax(m, gained(c, g[0], p));
      }
    }
    m = lanes_max64<64>(m);
    if constexpr (W > 1) {
      __syncthreads();
      if (lane == 0) part[wv] = m;
      __syncthreads();
      m = part[0];
#pragma unroll
      for (int i = 1; i < W; ++i) m = fmax(m, part[i]);
    }
    const NormScale s = norm_scale(m, inv, 127.0);
    if (tid == 0) a.scale[row] = s.stored;
    auto codes = [&](int c, const float* v) {
      gained(c, v, p);
      u32x2 o{0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = s.zero ? 0 : (int)fmin(fmax(rint(p[i] * s.mul), -127.0), 127.0);
        o[i / 4] |= ((uint32_t)k & 0xFFu) << (i % 4 * 8);
      }
      store8_codes<VEC>(static_cast<uint8_t*>(a.q) + row * H, c, H, o);
      if (a.out) put_out(c, p);
    };
    if constexpr (NC > 0) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (tid + T * i < chunks) codes(tid + T * i, g[i]);
    } else {
      for (int c = tid; c < chunks; c += T) {
        again(c, g[0]);
        codes(c, g[0]);
      }
    }
  }
}

template <int DT, bool F8>
static void norm_dt(NormArgs a, hipStream_t s) {
  auto at16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const bool one = a.rows == 1;
  const bool vec = a.hidden % 8 == 0 && at16(a.h) && at16(a.t) && at16(a.gain) && at16(a.h_out) && at16(a.out) &&
                   reinterpret_cast<uintptr_t>(a.q) % 8 == 0 && (one || a.h_stride % 4 == 0) &&
                   (one || !a.t || a.t_stride * Elem<DT>::bytes % 16 == 0);
  const int chunks = (a.hidden + kBlock - 1) / kBlock * kLanes;
  // a launch holds at most 2^31 threads: long calls go in pieces
  constexpr int kRows = 1 << 21;
  for (a.row0 = 0; a.row0 < a.rows; a.row0 += kRows) {
    const int n = a.rows - a.row0 < kRows ? a.rows - a.row0 : kRows;
#define NORM(VEC, T, NC, grid) \
  hipLaunchKernelGGL((k_norm_q<DT, F8, VEC, T, NC>), dim3(grid), dim3((T) < 256 ? 256 : (T)), 0, s, a)
    // A row a wave up to 1024 elements (65536 rows of 1024: 140 us, with 4 waves 164, 8 waves 261; of
    // 256: 50, 105, 206); above, 8 waves, or 16 where rows are few and time is latency (7168 elements, 1
    // row: 5.6 and 5.2 us, 2048 rows: 34.9 and 35.7, 16384 rows: 241 and 248; 4 waves 7.5, 39.8, 257).
    if (vec && chunks <= 128) NORM(true, 64, 2, (n + 3) / 4);
    else if (vec && chunks <= 1024 && n > 256) NORM(true, 512, 2, n);
    else if (vec && chunks <= 1024) NORM(true, 1024, 1, n);
    else if (vec) NORM(true, 1024, 0, n);
    else if (chunks <= 128) NORM(false, 64, 2, (n + 3) / 4);
    else if (chunks <= 1024) NORM(false, 512, 2, n);
    else NORM(false, 1024, 0, n);
#undef NORM
  }
}

hipError_t launch_norm_q(const NormArgs& a, int t_dtype, bool f8, hipStream_t s) {
#define NORM_DT(DT) (f8 ? norm_dt<DT, true>(a, s) : norm_dt<DT, false>(a, s))
  if (t_dtype == MOE_DTYPE_BF16) NORM_DT(MOE_DTYPE_BF16);
  else if (t_dtype == MOE_DTYPE_F16) NORM_DT(MOE_DTYPE_F16);
  else NORM_DT(MOE_DTYPE_F32);
#undef NORM_DT
  return hipGetLastError();
}

}  // namespace moe
