// api_common.h -- checks of arguments that the entry points share.
// Internal to libmoe_mxfp4.so.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "moe_mxfp4.h"

static inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
static inline bool float_dtype(moe_dtype t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F32 || t == MOE_DTYPE_F16; }
static inline size_t dtype_bytes(moe_dtype t) { return t == MOE_DTYPE_F32 ? 4 : t == MOE_DTYPE_I8 || t == MOE_DTYPE_F8 ? 1 : 2; }
static constexpr int kMaxI8K = 65536;  // 127 * 128 * k stays inside int32
static constexpr int kMaxCols = 1 << 20;
// What is written must not lie over what other workgroups still read.
static inline bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return a && b && p < q + b_bytes && q < p + a_bytes;
}
// The same for rows that may lie apart: whether the block touches one of them.
struct Rows {
  const void* base;
  size_t count, bytes, stride;  // bytes of a row, and from one to the next
};
static inline bool overlap(const Rows& r, const void* block, size_t bytes) {
  if (!overlap(r.base, (r.count - 1) * r.stride + r.bytes, block, bytes)) return false;
  const uintptr_t b = reinterpret_cast<uintptr_t>(r.base), q = reinterpret_cast<uintptr_t>(block);
  const size_t first = q < b + r.bytes ? 0 : (q - b - r.bytes) / r.stride + 1;  // row that ends behind the block's start
  return first < r.count && b + first * r.stride < q + bytes;
}

static inline bool slots_ok(int tokens, int top_k, int num_experts) {
  return tokens >= 1 && top_k >= 1 && top_k <= MOE_MAX_TOPK && num_experts >= 1 && num_experts <= MOE_MAX_EXPERTS &&
         (size_t)tokens * top_k < ((size_t)1 << 27);
}
