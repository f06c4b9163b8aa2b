// tile_device.h -- what the kernels of the 8-bit products share: the rows of a
// tile, loads straight to LDS, waits, the exchange before a store.  A is the
// argument block of a product (I8Args, F8Args).
// Internal to libmoe_mxfp4.so.
#pragma once

#include "i8_common.h"

namespace moe {

// The row that position p of a product reads and the one it writes.  Dense:
// both p.  Grouped: position p of the order names a slot, which is the row
// written; the row read is the slot (FC2) or its token (FC1)
// (clamped: whatever a groups buffer holds, no address leaves x or y).
template <class A>
__device__ __forceinline__ int y_row(const A& a, int p) {
  return a.order ? (int)min((unsigned)a.order[p], (unsigned)(a.rows - 1)) : p;
}
template <class A>
__device__ __forceinline__ int x_row(const A& a, int yr) { return a.x_div > 1 ? yr / a.x_div : yr; }

// The tile of rows a workgroup works on: expert, first position, positions.
struct Tile {
  int e, p0, rows;
};

template <int BM, class A>
__device__ __forceinline__ bool find_tile(const A& a, int t, Tile& o) {
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
// kernel of the integer products reached 4.3 TB/s that way.)
constexpr int KS = 128;

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void glb_void;

// 16 codes of zero: what a lane reads in place of codes of x past K.
static __device__ const __attribute__((aligned(16))) int8_t kZeroCodes[16] = {0};

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

}  // namespace moe
