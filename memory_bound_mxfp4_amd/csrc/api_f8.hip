// api_f8.hip -- the C entry points of the 8-bit floating-point operators and of
// the norms with an output in 8 bits: argument validation, workspaces, launches.
// Semantics are documented in moe_mxfp4.h.
#include <hip/hip_runtime.h>

#include <float.h>

#include "api_common.h"
#include "internal.h"
#include "moe_mxfp4.h"

using namespace moe;

static constexpr int kMaxK = 65536, kScaleBlock = 128;
static size_t blocks_of(int n) { return ((size_t)n + kScaleBlock - 1) / kScaleBlock; }

// The norms -----------------------------------------------------------------------

static moe_status norm_q(const float* h, size_t h_stride, const void* t, moe_dtype t_dtype, size_t t_stride,
                         const float* gain, int rows, int hidden, float eps, float* h_out, uint16_t* out, void* q,
                         float* scale, bool f8, void* stream) {
  if (!h || !q || !scale || rows < 1 || hidden < 1 || h_stride < (size_t)hidden || !(eps >= 0.0f) || !(eps <= FLT_MAX))
    return MOE_ERR_INVALID_ARGUMENT;
  if ((t != nullptr) != (h_out != nullptr)) return MOE_ERR_INVALID_ARGUMENT;
  if (t && (!float_dtype(t_dtype) || t_stride < (size_t)hidden || !aligned(t, dtype_bytes(t_dtype))))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(h, 4) || !aligned(gain, 4) || !aligned(h_out, 4) || !aligned(out, 2) || !aligned(scale, 4))
    return MOE_ERR_INVALID_ARGUMENT;
  if (hidden > kMaxK || rows > MOE_MAX_ROWS) return MOE_ERR_UNSUPPORTED;
  const size_t n = (size_t)rows, k = (size_t)hidden, ts = dtype_bytes(t_dtype);
  const Rows hr{h, n, 4 * k, 4 * h_stride}, tr{t, n, k * ts, t_stride * ts};
  // what is written: each apart from what is read and from the others; h_out may be h itself
  const struct {
    const void* p;
    size_t bytes;
  } to[4] = {{h_out, 4 * n * k}, {out, 2 * n * k}, {q, n * k}, {scale, 4 * n * (f8 ? blocks_of(hidden) : 1)}};
  for (int i = 0; i < 4; ++i) {
    if (!to[i].p) continue;
    const bool in_place = i == 0 && h_out == h && (rows == 1 || h_stride == k);
    if ((!in_place && overlap(hr, to[i].p, to[i].bytes)) || (t && overlap(tr, to[i].p, to[i].bytes)) ||
        overlap(gain, 4 * k, to[i].p, to[i].bytes))
      return MOE_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j)
      if (overlap(to[j].p, to[j].bytes, to[i].p, to[i].bytes)) return MOE_ERR_INVALID_ARGUMENT;
  }
  NormArgs a{};
  a.h = h;
  a.h_stride = h_stride;
  a.t = t;
  a.t_stride = t_stride;
  a.gain = gain;
  a.rows = rows;
  a.hidden = hidden;
  a.eps = eps;
  a.h_out = h_out;
  a.out = out;
  a.q = q;
  a.scale = scale;
  return launch_norm_q(a, t ? t_dtype : MOE_DTYPE_F32, f8, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK
                                                                                                           : MOE_ERR_HIP;
}

// The products --------------------------------------------------------------------

// The codes and scales of rows that a product quantises itself.
struct QuantWs {
  uint8_t* q;
  float* scale;
  size_t bytes;
};
static QuantWs quant_ws(void* ws, int rows, int k) {
  QuantWs w;
  const size_t codes = align256((size_t)rows * k);
  w.q = static_cast<uint8_t*>(ws);
  w.scale = reinterpret_cast<float*>(static_cast<char*>(ws) + codes);
  w.bytes = codes + align256(4 * rows * blocks_of(k));
  return w;
}

static moe_status check_f8(const void* x, moe_dtype x_dtype, size_t x_stride, const float* x_scale, int x_rows, int k,
                           const uint8_t* w, const float* w_scale, int n, int swiglu, const void* y, moe_dtype y_dtype,
                           size_t y_rows) {
  if (!x || !w || !w_scale || !y || x_rows < 1 || n < 1 || k < 16 || k % 16 || (swiglu != 0 && swiglu != 1))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!float_dtype(y_dtype) || !(float_dtype(x_dtype) || x_dtype == MOE_DTYPE_F8)) return MOE_ERR_INVALID_ARGUMENT;
  if ((x_dtype == MOE_DTYPE_F8) != (x_scale != nullptr) || x_stride < (size_t)k) return MOE_ERR_INVALID_ARGUMENT;
  if (x_dtype == MOE_DTYPE_F8 ? (!aligned(x, 16) || x_stride % 16) : !aligned(x, dtype_bytes(x_dtype)))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(w, 16) || !aligned(y, 16) || !aligned(w_scale, 4) || !aligned(x_scale, 4)) return MOE_ERR_INVALID_ARGUMENT;
  if (k > kMaxK || n > kMaxCols || x_rows > MOE_MAX_ROWS) return MOE_ERR_UNSUPPORTED;
  const size_t es = dtype_bytes(x_dtype);
  if (overlap(Rows{x, (size_t)x_rows, k * es, x_stride * es}, y, y_rows * n * dtype_bytes(y_dtype)))
    return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

// Whether a block that a product writes lies over its matrices, scales or groups.
static bool over_operands(const F8Args& a, const float* x_scale, int x_rows, const void* groups, size_t groups_bytes,
                          const void* block, size_t bytes) {
  const size_t matrices = (size_t)a.num_experts * (a.swiglu ? 2 : 1), kb = blocks_of(a.k);
  return overlap(a.w, matrices * a.n * a.k, block, bytes) ||
         overlap(a.w_scale, 4 * matrices * blocks_of(a.n) * kb, block, bytes) ||
         overlap(x_scale, 4 * (size_t)x_rows * kb, block, bytes) || overlap(groups, groups_bytes, block, bytes);
}
static size_t y_bytes(const F8Args& a) { return (size_t)a.rows * a.n * dtype_bytes((moe_dtype)a.y_dtype); }

// Workspace of a product: the codes and scales of rows it quantises, then the
// sums of a split K.
static size_t f8_ws_bytes(int x_rows, int k, moe_dtype x_dtype, const F8Plan& plan) {
  return (x_dtype == MOE_DTYPE_F8 ? 0 : quant_ws(nullptr, x_rows, k).bytes) + align256(plan.part_bytes);
}
// For outputs of any type.
static size_t f8_ws_size(int rows, int experts, bool grouped, int x_rows, int n, int k, int swiglu, moe_dtype x_dtype) {
  size_t most = 0;
  for (int wide = 0; wide < 2; ++wide) {
    const size_t b = f8_ws_bytes(x_rows, k, x_dtype, f8_plan(rows, experts, grouped, n, k, swiglu != 0, wide != 0));
    most = b > most ? b : most;
  }
  return most;
}

// Takes the workspace apart and quantises rows that are not codes already.
static moe_status f8_inputs(F8Args& a, const F8Plan& plan, const void* x, moe_dtype x_dtype, size_t x_stride,
                            const float* x_scale, int x_rows, int k, const void* groups, size_t groups_bytes, void* ws,
                            size_t ws_bytes, hipStream_t s) {
  a.x = static_cast<const int8_t*>(x);
  a.x_stride = x_stride;
  a.x_scale = x_scale;
  a.x_rows = x_rows;
  const size_t need = f8_ws_bytes(x_rows, k, x_dtype, plan);
  if (need && (!ws || !aligned(ws, 256))) return MOE_ERR_INVALID_ARGUMENT;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (over_operands(a, x_scale, x_rows, groups, groups_bytes, a.y, y_bytes(a))) return MOE_ERR_INVALID_ARGUMENT;
  if (!need) return MOE_OK;
  const size_t es = dtype_bytes(x_dtype);
  if (overlap(Rows{x, (size_t)x_rows, k * es, x_stride * es}, ws, need) || overlap(a.y, y_bytes(a), ws, need) ||
      over_operands(a, x_scale, x_rows, groups, groups_bytes, ws, need))
    return MOE_ERR_INVALID_ARGUMENT;
  char* p = static_cast<char*>(ws);
  if (x_dtype != MOE_DTYPE_F8) {
    const QuantWs w = quant_ws(p, x_rows, k);
    if (launch_quant_f8(x, x_dtype, x_stride, x_rows, k, w.q, w.scale, s) != hipSuccess) return MOE_ERR_HIP;
    a.x = reinterpret_cast<const int8_t*>(w.q);
    a.x_stride = (size_t)k;
    a.x_scale = w.scale;
    p += w.bytes;
  }
  a.parts = reinterpret_cast<float*>(p);
  return MOE_OK;
}

extern "C" {

moe_status quant_rows_f8(const void* x, moe_dtype dtype, size_t x_stride, int rows, int k, uint8_t* q, float* scale,
                         void* stream) {
  if (!x || !q || !scale || !float_dtype(dtype) || rows < 1 || k < 1 || x_stride < (size_t)k)
    return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(x, dtype_bytes(dtype)) || !aligned(scale, 4)) return MOE_ERR_INVALID_ARGUMENT;
  if (k > kMaxK || rows > MOE_MAX_ROWS) return MOE_ERR_UNSUPPORTED;
  const size_t es = dtype_bytes(dtype), codes = (size_t)rows * k, scales = 4 * rows * blocks_of(k);
  const Rows in{x, (size_t)rows, k * es, x_stride * es};
  if (overlap(in, q, codes) || overlap(in, scale, scales) || overlap(q, codes, scale, scales))
    return MOE_ERR_INVALID_ARGUMENT;
  if (launch_quant_f8(x, dtype, x_stride, rows, k, q, scale, static_cast<hipStream_t>(stream)) != hipSuccess)
    return MOE_ERR_HIP;
  return MOE_OK;
}

moe_status residual_add_rmsnorm_f8(const float* h, size_t h_stride, const void* t, moe_dtype t_dtype, size_t t_stride,
                                   const float* gain, int rows, int hidden, float eps, float* h_out, uint16_t* out,
                                   uint8_t* q, float* scale, void* stream) {
  return norm_q(h, h_stride, t, t_dtype, t_stride, gain, rows, hidden, eps, h_out, out, q, scale, true, stream);
}

moe_status residual_add_rmsnorm_i8(const float* h, size_t h_stride, const void* t, moe_dtype t_dtype, size_t t_stride,
                                   const float* gain, int rows, int hidden, float eps, float* h_out, uint16_t* out,
                                   int8_t* q, float* scale, void* stream) {
  return norm_q(h, h_stride, t, t_dtype, t_stride, gain, rows, hidden, eps, h_out, out, q, scale, false, stream);
}

size_t gemm_f8_workspace_size(int m, int n, int k, int swiglu, moe_dtype x_dtype) {
  if (m < 1 || n < 1 || k < 1 || m > MOE_MAX_ROWS || n > kMaxCols || k > kMaxK) return 0;
  return f8_ws_size(m, 1, false, m, n, k, swiglu, x_dtype);
}

moe_status gemm_f8(const void* x, moe_dtype x_dtype, size_t x_stride, const float* x_scale, int m, int k,
                   const uint8_t* w, const float* w_scale, int n, int swiglu, void* y, moe_dtype y_dtype, void* ws,
                   size_t ws_bytes, void* stream) {
  moe_status st = check_f8(x, x_dtype, x_stride, x_scale, m, k, w, w_scale, n, swiglu, y, y_dtype, m);
  if (st != MOE_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const F8Plan plan = f8_plan(m, 1, false, n, k, swiglu != 0, y_dtype == MOE_DTYPE_F32);
  const int tiles = (m + plan.tile_rows - 1) / plan.tile_rows;
  if (!f8_launchable(plan, n, swiglu != 0, tiles)) return MOE_ERR_UNSUPPORTED;
  F8Args a{};
  a.rows = m;
  a.k = k;
  a.n = n;
  a.w = reinterpret_cast<const int8_t*>(w);
  a.w_scale = w_scale;
  a.swiglu = swiglu != 0;
  a.y = y;
  a.y_dtype = y_dtype;
  a.num_experts = 1;
  a.x_div = 1;
  if (m == 1 && x_dtype != MOE_DTYPE_F8 && f8_token_ok(x, k, n, a.swiglu, 1)) {
    if (over_operands(a, nullptr, 1, nullptr, 0, y, y_bytes(a))) return MOE_ERR_INVALID_ARGUMENT;
    return launch_f8_token(a, x, x_dtype, 1, s) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
  }
  st = f8_inputs(a, plan, x, x_dtype, x_stride, x_scale, m, k, nullptr, 0, ws, ws_bytes, s);
  if (st != MOE_OK) return st;
  return launch_gemm_f8(a, plan, tiles, s) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

size_t experts_gemm_f8_workspace_size(int tokens, int top_k, int num_experts, int x_rows, int n, int k, int swiglu,
                                      moe_dtype x_dtype) {
  if (!slots_ok(tokens, top_k, num_experts) || x_rows < 1 || n < 1 || k < 1 || x_rows > MOE_MAX_ROWS ||
      n > kMaxCols || k > kMaxK)
    return 0;
  return f8_ws_size(tokens * top_k, num_experts, true, x_rows, n, k, swiglu, x_dtype);
}

moe_status experts_gemm_f8(const void* x, moe_dtype x_dtype, size_t x_stride, const float* x_scale, int x_rows, int k,
                           const void* groups, size_t groups_bytes, int tokens, int top_k, int num_experts,
                           const uint8_t* w, const float* w_scale, int n, int swiglu, void* y, moe_dtype y_dtype,
                           void* ws, size_t ws_bytes, void* stream) {
  if (!groups || !aligned(groups, 256) || !slots_ok(tokens, top_k, num_experts)) return MOE_ERR_INVALID_ARGUMENT;
  moe_status st = check_f8(x, x_dtype, x_stride, x_scale, x_rows, k, w, w_scale, n, swiglu, y, y_dtype,
                           (size_t)tokens * top_k);
  if (st != MOE_OK) return st;
  const size_t slots = (size_t)tokens * top_k;
  if (x_rows != tokens && (size_t)x_rows != slots) return MOE_ERR_INVALID_ARGUMENT;
  const GroupsLayout g = groups_layout(tokens, top_k, num_experts);
  if (groups_bytes < g.bytes) return MOE_ERR_WORKSPACE_TOO_SMALL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const F8Plan plan = f8_plan((int)slots, num_experts, true, n, k, swiglu != 0, y_dtype == MOE_DTYPE_F32);
  int map = 0;
  while (map + 1 < kTileMaps && kTileRows[map] != plan.tile_rows) ++map;
  if (!f8_launchable(plan, n, swiglu != 0, g.max_tiles[map])) return MOE_ERR_UNSUPPORTED;
  F8Args a{};
  const char* gp = static_cast<const char*>(groups);
  a.rows = (int)slots;
  a.k = k;
  a.n = n;
  a.w = reinterpret_cast<const int8_t*>(w);
  a.w_scale = w_scale;
  a.swiglu = swiglu != 0;
  a.y = y;
  a.y_dtype = y_dtype;
  a.num_experts = num_experts;
  a.x_div = (size_t)x_rows == slots ? 1 : top_k;
  a.order = reinterpret_cast<const int32_t*>(gp);
  if (x_rows == 1 && x_dtype != MOE_DTYPE_F8 && f8_token_ok(x, k, n, a.swiglu, g.max_tiles[0])) {
    if (over_operands(a, nullptr, 1, groups, g.bytes, y, y_bytes(a))) return MOE_ERR_INVALID_ARGUMENT;
    a.num_tiles = reinterpret_cast<const int32_t*>(gp + g.counts);
    a.tiles = reinterpret_cast<const int2*>(gp + g.tiles[0]);
    return launch_f8_token(a, x, x_dtype, g.max_tiles[0], s) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
  }
  a.num_tiles = reinterpret_cast<const int32_t*>(gp + g.counts) + map;
  a.tiles = reinterpret_cast<const int2*>(gp + g.tiles[map]);
  st = f8_inputs(a, plan, x, x_dtype, x_stride, x_scale, x_rows, k, groups, g.bytes, ws, ws_bytes, s);
  if (st != MOE_OK) return st;
  return launch_gemm_f8(a, plan, g.max_tiles[map], s) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
