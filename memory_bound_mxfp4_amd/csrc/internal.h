// internal.h -- host-side launchers and the workspace layout shared by the
// library's translation units.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_mxfp4.h"

namespace moe {

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Offsets of the six sub-arrays of an expert blob (layout documented in
// moe_mxfp4.h): gate codes, up codes, down codes, gate/up/down scales.
struct BlobLayout {
  size_t off[6];
  size_t bytes;
};
BlobLayout blob_layout(int H, int I);

// Expert-gathered schedule built on the device from the top-k indices.
//   active[U]         the U distinct experts any row selected, ascending
//   row_off[U+1]      rows of active expert a are rows[row_off[a] .. row_off[a+1])
//   rows[B*k]         slot ids s = b * k + j
//   cg_off[U+1]       batch > 1: active expert a has column groups (up to 16
//                     of its rows each) cg_off[a] .. cg_off[a+1]
struct Sched {
  int* cg_off;
  int* active;
  int* row_off;
  int* rows;
};

// Control block at the start of the workspace: uint32 words, each counter on
// a 128-byte line of its own (line i starts at word CTRL_STRIDE * i) so that
// polls of different counters never share a cache line.
//   line 0, word 0   head of work queue 0           (zero between calls)
//   line 0, word 7   sticky error word (byte offset MOE_WS_STATUS_OFFSET)
//   line 1           workgroups that have exited    (zero between calls)
//   line 2           call epoch: bumped by the last workgroup of every call
//   line 3           schedule-ready word pair (batch > 1): U | tag << 32
//   line 4           head of work queue 1           (zero between calls)
// Data handed between workgroups inside a call travels as 8-byte pairs
// (32-bit value | 32-bit tag << 32), tag = epoch + 1 of the call, written and
// read with single 8-byte coherent accesses: a consumer polls the data itself
// until every pair carries its call's tag, so no producer ever has to drain
// its stores and bump a counter.
constexpr int CTRL_STRIDE = 32;
constexpr int CTRL_HEAD = 0, CTRL_ERR = 7, CTRL_EXIT = 1 * CTRL_STRIDE, CTRL_EPOCH = 2 * CTRL_STRIDE,
              CTRL_READY = 3 * CTRL_STRIDE, CTRL_HEAD1 = 4 * CTRL_STRIDE, CTRL_WORDS = 5 * CTRL_STRIDE;

// Workspace of moe_decode_layer.
struct Workspace {
  unsigned* ctrl;
  int umax;
  uint64_t* logits_p;  // [B][E]      router logits
  uint64_t* idx_p;     // [B*k]       expert of slot s = b*k + j
  uint64_t* gate_p;    // [B*k]       gate of slot s
  Sched sched;         // batch > 1: expert-gathered schedule (plain ints, published by READY)
  uint64_t* hs_p;      // [B][Is]     shared-expert SwiGLU output
  uint64_t* hr_p;      // [B*k][I]    routed SwiGLU output, by slot
  uint64_t* os_p;      // [B][H]      shared-expert output
  uint64_t* or_p;      // [B*k][H]    routed expert outputs, by slot
  uint64_t* hflag;     // batch > 1: [umax + 1][4][hflag_tiles] "FC1 tile done" tags
  int hflag_tiles;
  size_t bytes;
};
Workspace ws_layout(void* base, int H, int I, int E, int k, int Is, int B);

// ---- launchers (return hipSuccess or the launch error) ----
hipError_t launch_router_logits(const uint16_t* x, int B, int H, const uint16_t* wr, const float* bias, int E,
                                float* logits, hipStream_t s);
hipError_t launch_topk(const float* logits, int B, int E, int k, int32_t* idx, float* gate, hipStream_t s);

struct LayerArgs {
  int H, I, E, k, Is, B;
  const uint16_t* x;
  const uint16_t *sg, *su, *sd;
  const uint8_t* experts;
  BlobLayout blob;
  const float* gate;
  Workspace ws;
  float* residual;
};
// mx8: the routed experts' FP4 x MXFP8 variant (the matrix-core kernel at
// every batch); mx8_supported: the shapes that variant covers.
hipError_t launch_layer(const LayerArgs& a, const float* bias, const uint16_t* wr, int32_t* idx, hipStream_t s,
                        bool mx8 = false);
bool mx8_supported(int H, int I);
// Cap on the layer kernel's grid (0: two workgroups per compute unit).
void set_layer_grid_cap(int n);
hipError_t launch_zero(void* p, size_t bytes, hipStream_t s);
hipError_t launch_pack_experts(uint8_t* experts, int E, int H, int I, uint8_t* scratch, bool to_packed,
                               hipStream_t s);

hipError_t launch_gemv_mxfp4(const uint8_t* codes, const uint8_t* scales, int N, int K, const void* x, bool x_f32,
                             int B, float* y, hipStream_t s);

hipError_t launch_rmsnorm(const float* in, int B, int H, float eps, uint16_t* out, hipStream_t s);
hipError_t launch_dense_gemv(const uint16_t* w, int N, int K, const uint16_t* x, int B, uint16_t* y, hipStream_t s);
hipError_t launch_residual_add(float* h, const uint16_t* t, int B, int H, hipStream_t s);
hipError_t launch_residual_add_rmsnorm(float* h, const uint16_t* t, int B, int H, float eps, uint16_t* out,
                                       hipStream_t s);

hipError_t launch_stream_read(const void* buf, size_t bytes, int blocks_per_cu, uint32_t* sink, hipStream_t s);
hipError_t launch_prefetch(const moe_range* ranges, int n, int blocks, hipStream_t s);

// ---- routing, slots by expert, 8-bit products ----
hipError_t launch_route(const void* logits, int dtype, size_t row_stride, int rows, const float* bias,
                        const moe_route_params& p, int32_t* idx, float* gate, hipStream_t s);

// A slot-groups buffer: order at byte 0, then offsets, the number of tiles of
// each map, and the maps.  Map i lists, for every expert that has slots (and
// for the slots without one, as expert num_experts), the tiles of kTileRows[i]
// of its positions: {expert | positions << 16, first position}.
constexpr int kTileMaps = 4;
constexpr int kTileRows[kTileMaps] = {16, 64, 128, 256};
// The most tiles of that many rows that slots of so many experts make: whole ones, and an end of each expert.
inline int max_tiles(size_t slots, int num_experts, int tile_rows) {
  const size_t ends = (size_t)num_experts + 1;
  return (int)(slots / tile_rows + (slots < ends ? slots : ends));
}
struct TileMaps {
  int2* t[kTileMaps];
};
struct GroupsLayout {
  size_t offsets, counts, tiles[kTileMaps], hist;
  int max_tiles[kTileMaps];
  int blocks;  // workgroups of the sort
  size_t bytes;
};
GroupsLayout groups_layout(int tokens, int top_k, int E);
hipError_t launch_group_slots(const int32_t* idx, int tokens, int top_k, int E, void* groups, hipStream_t s);
hipError_t launch_combine(const void* y, int dtype, const float* gate, int tokens, int top_k, int H,
                          const float* residual, float* out, hipStream_t s);

hipError_t launch_quant_rows(const void* x, int dtype, size_t x_stride, int rows, int K, int8_t* q, float* scale,
                             hipStream_t s);

struct I8Args {
  const int8_t* x;
  size_t x_stride;
  const float* x_scale;
  int rows, k, n;  // rows: positions of the product (dense rows, or slots)
  const int8_t* w;
  const float* w_scale;
  bool swiglu;
  void* y;
  int y_dtype;
  // grouped products; order NULL: dense
  const int32_t *order, *num_tiles;
  const int2* tiles;
  int num_experts, x_div;
  int32_t* parts;  // int32 sums of each part of a split K: [part][position][columns of all tiles]
};
// How a product runs: kernel and tile (kind), rows of a tile, parts that K is
// split into and the bytes of their sums.  rows: dense rows, or slots of
// `experts` experts.
struct I8Plan {
  int kind, tile_rows, parts;
  size_t part_bytes;
};
I8Plan i8_plan(int rows, int experts, bool grouped, int n, int k, bool swiglu);
// A product of one float row that the kernel quantises itself, on the tiles of
// 16 positions; i8_token_ok: the rows it takes.
bool i8_token_ok(const void* x, int dtype, int k, int n, bool swiglu, int max_tiles);
hipError_t launch_i8_token(const I8Args& a, const void* x, int dtype, int max_tiles, hipStream_t s);
// Whether the launch of a plan stays inside the size of a grid.
bool i8_launchable(const I8Plan& plan, int n, bool swiglu, int max_tiles);
hipError_t launch_gemm_i8(const I8Args& a, const I8Plan& plan, int max_tiles, hipStream_t s);

// ---- 8-bit floating point ----
hipError_t launch_quant_f8(const void* x, int dtype, size_t x_stride, int rows, int K, uint8_t* q, float* scale,
                           hipStream_t s);

struct NormArgs {
  const float* h;
  size_t h_stride;
  const void* t;  // NULL: nothing is added, and h_out is not written
  size_t t_stride;
  const float* gain;  // NULL: ones
  int rows, row0, hidden;
  float eps;
  float* h_out;
  uint16_t* out;  // the normalised rows in bf16, or NULL
  void* q;
  float* scale;
};
hipError_t launch_norm_q(const NormArgs& a, int t_dtype, bool f8, hipStream_t s);

struct F8Args {
  const int8_t* x;
  size_t x_stride;
  const float* x_scale;  // [blocks of K][x_rows]
  int x_rows;
  int rows, k, n;  // rows: positions of the product (dense rows, or slots)
  const int8_t* w;
  const float* w_scale;  // of each matrix [blocks of n][blocks of K]
  bool swiglu;
  void* y;
  int y_dtype;
  // grouped products; order NULL: dense
  const int32_t *order, *num_tiles;
  const int2* tiles;
  int num_experts, x_div;
  float* parts;  // sums of each part of a split K: [part][position][columns of all tiles]
};
// How a product runs, as I8Plan; wide: products in fp16 (outputs of fp32).
struct F8Plan {
  int kind, tile_rows, parts;
  size_t part_bytes;
};
F8Plan f8_plan(int rows, int experts, bool grouped, int n, int k, bool swiglu, bool wide);
// A product of one float row that the kernel quantises itself, on the tiles of
// 16 positions; f8_token_ok: the rows it takes.
bool f8_token_ok(const void* x, int k, int n, bool swiglu, int max_tiles);
hipError_t launch_f8_token(const F8Args& a, const void* x, int dtype, int max_tiles, hipStream_t s);
bool f8_launchable(const F8Plan& plan, int n, bool swiglu, int max_tiles);
hipError_t launch_gemm_f8(const F8Args& a, const F8Plan& plan, int max_tiles, hipStream_t s);

int num_cus();

}  // namespace moe
