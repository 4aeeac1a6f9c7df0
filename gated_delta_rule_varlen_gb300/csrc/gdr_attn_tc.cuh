// gdr_attn_tc.cuh -- pieces of the attention kernels on the tensor cores.
#pragma once
#include <algorithm>

#include "gdr_attn.cuh"
#include "gdr_tc_roles.cuh"

namespace gdr {

constexpr int TILE = 128;  // rows of a tile of queries or keys

// The key tiles [lo, hi) that tokens [i0, i1) of a document see.
struct TileRange {
  int lo, hi;
};
__device__ __forceinline__ TileRange tiles_of(const AttnArgs& a, const AttnBlock& b, int i0, int i1) {
  if (i0 >= i1) return {0, 0};
  const KeyRange first = keys_of(a, i0, b.lq, b.lk), last = keys_of(a, i1 - 1, b.lq, b.lk);
  if (last.hi <= first.lo) return {0, 0};
  return {first.lo / TILE, (last.hi + TILE - 1) / TILE};
}

template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N]) {  // nothing that reads them moves before this
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Whether the kernels take the arguments: what TMA addresses, and tiles of up to 128 columns.
inline bool attn_tc_shape(int D) { return D % 8 == 0 && D <= 128; }

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

// Heads that share their keys lie side by side in a tile of queries (row r is token r >> pack,
// head r & (2^pack - 1)) while the longest document's queries alone do not fill it.
inline int attn_pack(const AttnArgs& a, const int32_t* cu) {
  int most = 0, pack = 0;
  for (int i = 0; i < a.N; ++i) most = std::max(most, cu[i + 1] - cu[i]);
  const int G = a.H / a.HK;
  while (pack < 7 && G % (2 << pack) == 0 && ((int64_t)most << pack) < TILE) ++pack;
  return pack;
}

}  // namespace gdr
