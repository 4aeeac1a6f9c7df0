// gdr_norm.cuh -- the norms around a block, fused with its gate and residual:
//   u = x                          or  x r1 w_post,  r1 = (mean x^2 + eps)^(-1/2)
//   u = u act(z)                   with a gate z: act = silu or sigmoid
//   h = residual + alpha u         or  u
//   y = h r2 w,                    r2 = (mean h^2 + eps)^(-1/2)
// Every step is optional.  A row (of D elements) is held in registers by TPR
// threads from its one read to its one write; the means are FP32 sums by
// shuffles (and across warps through shared memory) in a fixed order.
#pragma once
#include "gdr_ops.cuh"
#include "gdr_runtime.h"

namespace gdr {

struct RowTensor {
  const void* p;
  int64_t s0, s1;  // element strides of the two leading dimensions
};

struct NormArgs {
  int64_t rows;  // R0 * R1
  int R1, D;
  RowTensor x, gate, res;  // gate.p, res.p null when absent
  const void *w_post, *w;  // [D] or null
  int wf32;
  int sigmoid;             // act: 0 silu, 1 sigmoid
  float alpha, eps;
  void *h, *y;             // outputs, dense [rows][D], or null
  // backward
  RowTensor dh, dy;        // or null
  void *dx, *dgate, *dres; // dense, or null
  float* part;             // [blocks][2][D]: partial dw, dw_post
};

// What a call needs decides the path: the smallest power-of-two group of
// threads that holds the row, NV vectors of V elements each.
struct NormShape {
  int V, TPR, NV;
};

cudaError_t launch_norm_fwd(const NormArgs& a, int dtype, const NormShape& s, int blocks, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormArgs& a, int dtype, const NormShape& s, int blocks, cudaStream_t st);

// Threads in a block of a shape: 128 for the shapes of up to a warp a row.
constexpr int norm_threads(int TPR) { return TPR < 128 ? 128 : TPR; }

template <int TPR>
struct RowGroup {
  static constexpr int THREADS = norm_threads(TPR);
  static constexpr int GROUPS = THREADS / TPR;  // rows a block works on at a time
  static constexpr int WARPS = TPR > 32 ? TPR / 32 : 1;

  // Sums of a and b over the row's threads, on every thread of the row.
  static __device__ __forceinline__ void sum2(float& a, float& b, float2* sm) {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int m = W / 2; m >= 1; m >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, m);
      b += __shfl_xor_sync(0xffffffffu, b, m);
    }
    if constexpr (TPR > 32) {
      // two buffers in turn, so that one barrier per sum is enough
      const int warp = threadIdx.x >> 5;
      if ((threadIdx.x & 31) == 0) sm[warp] = make_float2(a, b);
      __syncthreads();
      a = 0.f;
      b = 0.f;
#pragma unroll
      for (int i = 0; i < WARPS; ++i) {
        const float2 v = sm[i];
        a += v.x;
        b += v.y;
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ const T* row_ptr(const RowTensor& t, int64_t r, int R1) {
  const int64_t i = r / R1;
  return static_cast<const T*>(t.p) + i * t.s0 + (r - i * R1) * t.s1;
}

}  // namespace gdr
