// gdr_attn.cuh -- softmax attention over packed documents: arguments and pieces that
// its kernels share.  Per document with lq queries and lk keys (its own lk - lq keys
// come before its first query), query i sees the keys
//   j < lk,   j <= i + lk - lq (causal),   j > i + lk - lq - window (window > 0)
//   s_ij = scale q_i . k_j,  lse_i = log sum_j e^s_ij,  p_ij = e^(s_ij - lse_i),
//   out_i = sum_j p_ij v_j.
// Backward, with dp_ij = dout_i . v_j and delta_i = sum_j p_ij dp_ij = dout_i . out_i:
//   dv_j = sum_i p_ij dout_i,  ds_ij = p_ij (dp_ij - delta_i),
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,
// dk and dv summed over the H / HK query heads that share a key head.
#pragma once
#include <cuda.h>
#include "gdr_ops.cuh"
#include "gdr_runtime.h"

namespace gdr {

// [tokens][heads][D], dense rows: element strides of a token and of a head.
struct AttnRows {
  const __nv_bfloat16* p;
  int64_t s0, s1;
  __device__ __forceinline__ const __nv_bfloat16* row(int64_t t, int h) const { return p + t * s0 + h * s1; }
};

constexpr int ATTN_ORDERED = 256;
struct AttnArgs {
  AttnRows q, k, v, dout;
  const int *cu, *cuk;       // documents' queries and keys
  int N, H, HK, D;
  int64_t T, TK;
  float scale;
  int causal, window;
  __nv_bfloat16* out;        // [T][H][D]
  float* lse;                // [H][T]
  const __nv_bfloat16* o;    // backward: the forward's out and lse
  const float* lse_in;
  float* delta;              // [H][T]
  __nv_bfloat16 *dq, *dk, *dv;
  // The documents, those with the most keys first (their blocks are the longest), where there
  // are few enough of them.
  int ordered;
  uint8_t order[ATTN_ORDERED];
};

// The keys [lo, hi) that a query sees.
struct KeyRange {
  int lo, hi;
};
__host__ __device__ __forceinline__ KeyRange keys_of(const AttnArgs& a, int i, int lq, int lk) {
  KeyRange r{0, lk};
  const int last = i + lk - lq;  // (its own place)
  if (a.causal && last < lk) r.hi = last + 1;
  if (a.window && last >= a.window) r.lo = last - a.window + 1;
  return r;
}

// Blocks of `per` queries or keys of a document, those with the most work under a causal mask
// first: the later queries (LAST) or the earlier keys.
struct AttnBlock {
  int first;           // token within the document
  int q0, lq, k0, lk;  // the document's queries and keys
};
// Finds blocks of the documents (one warp, the same answer on every lane): 32 documents are held
// in registers, and the search goes on from them, or from the first ones for a block before them
// (blocks taken over come in no order that the hardware promises).
template <bool LAST>
struct BlockFinder {
  const AttnArgs& a;
  const int per;
  int before = 0;  // the blocks of the documents before d0
  int d0, q0, lq, k0, lk, n, pre, total;  // documents d0 + lane, their blocks, the sum up to them, of all 32

  __device__ __forceinline__ BlockFinder(const AttnArgs& args, int per_) : a(args), per(per_) { load(0); }
  __device__ __forceinline__ void load(int first) {
    const int lane = threadIdx.x & 31;
    int d = first + lane;
    d0 = first;
    q0 = lq = k0 = lk = 0;
    const bool is = d < a.N;
    if (is) {
      if (a.ordered) d = a.order[d];
      q0 = a.cu[d];
      lq = a.cu[d + 1] - q0;
      k0 = a.cuk[d];
      lk = a.cuk[d + 1] - k0;
    }
    n = is ? ((LAST ? lq : lk) + per - 1) / per : 0;
    pre = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, pre, m);
      if (lane >= m) pre += v;
    }
    total = __shfl_sync(0xffffffffu, pre, 31);
  }
  __device__ __forceinline__ AttnBlock find(int want) {
    if (want < before) {
      before = 0;
      load(0);
    }
#pragma unroll 1
    while (want - before >= total && d0 + 32 < a.N) {
      before += total;
      load(d0 + 32);
    }
    want -= before;
    const int l = __ffs(__ballot_sync(0xffffffffu, want < pre)) - 1;
    if (l < 0) return AttnBlock{0, 0, 0, 0, 0};  // (no document has it)
    AttnBlock b;
    const int end = __shfl_sync(0xffffffffu, pre, l);  // of the document's blocks
    b.first = (LAST ? end - 1 - want : want - end + __shfl_sync(0xffffffffu, n, l)) * per;
    b.q0 = __shfl_sync(0xffffffffu, q0, l);
    b.lq = __shfl_sync(0xffffffffu, lq, l);
    b.k0 = __shfl_sync(0xffffffffu, k0, l);
    b.lk = __shfl_sync(0xffffffffu, lk, l);
    return b;
  }
};

// How the kernels on the tensor cores cut the work: heads side by side in a tile of queries
// (2^pack), and into how many parts the sums of each kernel's blocks, joined by another
// kernel from scratch.
struct AttnPlan {
  int pack, fwd, dq, dkv;
  size_t fwd_bytes, bwd_bytes;
};
bool attn_tc_shape(int D);
AttnPlan attn_plan(const AttnArgs& a, const int32_t* cu, const int32_t* cuk);  // cu, cuk: the host's

cudaError_t launch_attn_fwd(const AttnArgs& a, const AttnPlan& p, const int32_t* cu, const int32_t* cuk, float* scratch,
                            cudaStream_t st);
cudaError_t launch_attn_bwd(const AttnArgs& a, const AttnPlan& p, const int32_t* cu, const int32_t* cuk, float* scratch,
                            cudaStream_t st);

}  // namespace gdr
