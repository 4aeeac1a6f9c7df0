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
};

// The keys [lo, hi) that a query sees.
struct KeyRange {
  int lo, hi;
};
__device__ __forceinline__ KeyRange keys_of(const AttnArgs& a, int i, int lq, int lk) {
  KeyRange r{0, lk};
  if (a.causal) r.hi = min(lk, i + lk - lq + 1);
  if (a.window && i + lk - lq >= a.window) r.lo = i + lk - lq - a.window + 1;
  return r;
}

}  // namespace gdr
