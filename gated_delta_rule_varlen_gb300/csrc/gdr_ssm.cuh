// gdr_ssm.cuh -- arguments and pieces that the selective scan's kernels share.
#pragma once
#include <cuda.h>
#include "gdr_ops.cuh"
#include "gdr_runtime.h"

namespace gdr {

struct SsmArgs {
  const __nv_bfloat16* x;
  int64_t ldx;
  const void* dt;
  int dt_f32;
  int64_t lddt;
  const float* A;
  const __nv_bfloat16 *B, *C;
  int64_t ldb, ldc;
  const float *D, *dt_bias;  // [H] or null
  int softplus;
  const int* cu;
  int N, T, H, P, G, NS;  // documents, tokens, heads, head dim, groups, state size
  const float* h0;        // [N][H][NS][P] or null
  __nv_bfloat16* out;     // [T][H][P]
  float* ht;              // [N][H][NS][P] or null
  // step
  float* state;           // [S][H][NS][P]
  const int* slots;
  int S;
};

// log(1 + e^x) = max(x, 0) + log(1 + y) with y = e^-|x| in (0, 1], and log(1 + y)
// = 2 atanh(t), t = y / (2 + y) <= 1/3, by its series 2 t (1 + t^2/3 + t^4/5 +
// ...), whose first seven terms leave less than 2^-26; small y keep their
// relative accuracy.  The exponent's product with log2(e) carries its rounding
// error along (as the factor 1 + err ln 2).
__device__ __forceinline__ float softplus_f(float x) {
  const float z = fminf(fabsf(x), 1e4f), e = -z * LOG2E;  // e^-1e4 is 0 (and inf stays out of the products)
  const float err = fmaf(-z, LOG2E, -e) - z * 1.92596299e-8f;  // log2(e) - LOG2E
  const float y = ex2(e) * fmaf(err, 0.69314718f, 1.f);
  const float t = __fdividef(y, 2.f + y), t2 = t * t;
  float s = fmaf(t2, 1.f / 13.f, 1.f / 11.f);
  s = fmaf(t2, s, 1.f / 9.f);
  s = fmaf(t2, s, 1.f / 7.f);
  s = fmaf(t2, s, 1.f / 5.f);
  s = fmaf(t2, s, 1.f / 3.f);
  s = fmaf(t2, s, 1.f);
  const float v = fmaxf(x, 0.f) + 2.f * t * s;
  return x != x ? x : v;
}

__device__ __forceinline__ float load_dt(const SsmArgs& a, int64_t t, int h) {
  float v = a.dt_f32 ? static_cast<const float*>(a.dt)[t * a.lddt + h]
                     : to_f(static_cast<const __nv_bfloat16*>(a.dt)[t * a.lddt + h]);
  if (a.dt_bias) v += a.dt_bias[h];
  return a.softplus ? softplus_f(v) : v;
}

// The chunked scan on the tensor cores (gdr_ssm_tc.cu): whether these
// arguments can take it, how it cuts the documents, its scratch and its launch.
struct SsmPlan {
  int lseg;          // chunks of a segment at most
  int64_t nseg;      // segments of all documents (an empty document has one)
  int64_t states;    // segments of documents that have several
  int64_t chunks;    // chunks of all documents (an empty document has one)
  bool split;        // some document has several
  size_t scratch;    // bytes
};
bool ssm_tc_shape(int P, int NS);
bool ssm_tc_layout(const SsmArgs& a);
SsmPlan ssm_tc_plan(int H, int P, int NS, int G, int N, const int32_t* cu_host);
cudaError_t launch_ssm_tc(const SsmArgs& a, const SsmPlan& plan, void* scratch, cudaStream_t st);

}  // namespace gdr
