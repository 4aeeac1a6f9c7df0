// gdr_attn_tc.cuh -- pieces of the attention kernels on the tensor cores.
#pragma once
#include <algorithm>

#include "gdr_attn.cuh"
#include "gdr_tc_roles.cuh"

namespace gdr {

constexpr int TILE = 128;  // rows of a tile of queries or keys

// The tiles [lo, hi) that a block goes through.
struct TileRange {
  int lo, hi;
};
// Of keys: those that queries [i0, i1) of a document see.
__host__ __device__ __forceinline__ TileRange tiles_of(const AttnArgs& a, int lq, int lk, int i0, int i1) {
  if (i0 >= i1) return {0, 0};
  const KeyRange first = keys_of(a, i0, lq, lk), last = keys_of(a, i1 - 1, lq, lk);
  if (last.hi <= first.lo) return {0, 0};
  return {first.lo / TILE, (last.hi + TILE - 1) / TILE};
}
// Of queries, `tokens` a tile: those that see any of the keys [first, last].
__host__ __device__ __forceinline__ TileRange query_tiles_of(const AttnArgs& a, int lq, int lk, int first, int last, int tokens) {
  const int off = lk - lq;
  const int lo = a.causal && first > off ? first - off : 0;
  int hi = lq;
  if (a.window && (int64_t)last - off + a.window < lq) hi = last - off + a.window;
  if (hi <= lo) return {0, 0};
  return {lo / tokens, (hi + tokens - 1) / tokens};
}
// Part `part` of `parts` of a range.
__device__ __forceinline__ TileRange part_of(const TileRange& r, int part, int parts) {
  const int64_t n = r.hi - r.lo;
  return {r.lo + (int)(n * part / parts), r.lo + (int)(n * (part + 1) / parts)};
}

template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N]) {  // nothing that reads them moves before this
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Whether TMA addresses the tensors.
inline bool attn_tc_layout(const AttnArgs& a) {
  for (const AttnRows* t : {&a.q, &a.k, &a.v, &a.dout})
    if (t->p && (((uintptr_t)t->p & 15) != 0 || t->s0 <= 0 || t->s1 <= 0 || t->s0 % 8 != 0 || t->s1 % 8 != 0)) return false;
  for (const void* p : {(const void*)a.out, (const void*)a.o, (const void*)a.dq, (const void*)a.dk, (const void*)a.dv})
    if (((uintptr_t)p & 15) != 0) return false;
  return true;
}

// [T][heads][D] BF16: boxes of 64 elements x `heads` heads x `tokens` tokens, 128-byte
// swizzle, zero fill outside.
inline bool attn_map(CUtensorMap* map, const AttnRows& t, int64_t T, int H, int D, int heads, int tokens) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  cuuint64_t strides[2] = {(cuuint64_t)t.s1 * 2, (cuuint64_t)t.s0 * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(t.p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gdr
