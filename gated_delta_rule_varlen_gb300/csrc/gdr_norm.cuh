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
#include <algorithm>

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
  int wvec;                // the weights can be read like the rows
  int sigmoid;             // act: 0 silu, 1 sigmoid
  float alpha, eps;
  void *h, *y;             // outputs, dense [rows][D], or null
  // backward
  RowTensor dh, dy;        // or null
  void *dx, *dgate, *dres; // dense, or null
  float* part;             // [blocks][2][D]: partial dw, dw_post
};

// The threads of a row: TPR of them with NV vectors of V elements each.
struct NormShape {
  int V, TPR, NV;
};

cudaError_t launch_norm_fwd(const NormArgs& a, int dtype, const NormShape& s, cudaStream_t st);
// *blocks: how many blocks ran (and left a partial row each)
cudaError_t launch_norm_bwd(const NormArgs& a, int dtype, const NormShape& s, int* blocks, cudaStream_t st);

// Most blocks of an SM that a backward is launched with, by threads of a block.
constexpr int norm_blocks_per_sm(int threads) { return threads <= 128 ? 8 : threads <= 256 ? 4 : threads <= 512 ? 2 : 1; }

// Threads in a block of a shape: 128 for the shapes of up to a warp a row.
constexpr int norm_threads(int TPR) { return TPR < 128 ? 128 : TPR; }

// As many blocks as the GPU holds at a time (each goes through its share of the
// rows), or fewer where there are fewer rows.
template <typename K>
int norm_grid(K kernel, int threads, size_t smem, int64_t groups, int occ_limit, int* occ_cache) {
  if (*occ_cache == 0) {
    int occ = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, threads, smem) != cudaSuccess || occ < 1) occ = 1;
    *occ_cache = occ;
  }
  const int64_t most = (int64_t)152 * std::min(*occ_cache, occ_limit);
  return (int)std::min<int64_t>(groups, most);
}

template <int TPR>
struct RowGroup {
  static constexpr int THREADS = norm_threads(TPR);
  static constexpr int GROUPS = THREADS / TPR;  // rows a block works on at a time
  static constexpr int WARPS = TPR > 32 ? TPR / 32 : 1;

  // Sum of a over the row's threads, on every thread of the row.
  static __device__ __forceinline__ void sum(float& a, float2* sm) {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int m = W / 2; m >= 1; m >>= 1) a += __shfl_xor_sync(0xffffffffu, a, m);
    if constexpr (TPR > 32) {
      const int warp = threadIdx.x >> 5;
      if ((threadIdx.x & 31) == 0) sm[warp].x = a;
      __syncthreads();
      a = 0.f;
#pragma unroll
      for (int i = 0; i < WARPS; ++i) a += sm[i].x;
    }
  }
  static __device__ __forceinline__ void sum2(float& a, float& b, float2* sm) {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int m = W / 2; m >= 1; m >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, m);
      b += __shfl_xor_sync(0xffffffffu, b, m);
    }
    if constexpr (TPR > 32) {
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

// The rows of a thread, every `step`-th one, in up to K tensors: their addresses
// advance by one sum, and another where the inner index wraps, without a
// multiplication or division a row.
template <typename T, int K>
struct Cursor {
  int64_t r, step;   // row
  int i1, step1, R1; // inner index
  const T* p[K];     // the tensors' rows
  int64_t by[K], wrap[K];
  __device__ __forceinline__ Cursor(int64_t first, int64_t step_, int R1_) : r(first), step(step_), R1(R1_) {
    i1 = (int)(first % R1);
    step1 = (int)(step % R1);
  }
  __device__ __forceinline__ void add(int k, const RowTensor& t) {
    p[k] = static_cast<const T*>(t.p) + (r / R1) * t.s0 + i1 * t.s1;
    by[k] = (step / R1) * t.s0 + step1 * t.s1;
    wrap[k] = t.s0 - R1 * t.s1;
  }
  __device__ __forceinline__ void next() {
    r += step;
    i1 += step1;
    const bool over = i1 >= R1;
    if (over) i1 -= R1;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      p[k] += by[k];
      if (over) p[k] += wrap[k];
    }
  }
};

// The rows a thread works on next, asked for DEPTH rows ahead: ITEMS vectors of
// the thread a row, in shared memory (gdr_ops.cuh: RowRing).
template <typename T, int V, int ITEMS, int DEPTH, int THREADS>
struct RowsAhead {
  static constexpr int BYTES = DEPTH * ITEMS * THREADS * (int)sizeof(Vec<T, V>);
  RowRing<T, V, DEPTH * ITEMS, THREADS> ring;
  __device__ __forceinline__ explicit RowsAhead(void* smem) : ring(smem) {}
  __device__ __forceinline__ void ask(int slot, int item, const T* src) { ring.push(slot * ITEMS + item, src, true); }
  __device__ __forceinline__ Vec<T, V> get(int slot, int item) const { return ring.at(slot * ITEMS + item); }
};

// V elements of a weight from c on, in pairs.
template <typename T, int V>
__device__ __forceinline__ void load_weight(const NormArgs& a, const void* p, int c, uint64_t (&f)[pairs_of<V>]) {
  if (V > 1 && a.wvec) {
    if (a.wf32) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const ulonglong2 v = __ldg(reinterpret_cast<const ulonglong2*>(static_cast<const float*>(p) + c + 4 * i));
        f[2 * i] = v.x;
        f[V > 1 ? 2 * i + 1 : 0] = v.y;
      }
    } else {
      to_pairs<T, V>(vload<T, V>(static_cast<const T*>(p) + c), f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < pairs_of<V>; ++i)
      f[i] = pack2(load_param<T>(p, a.wf32, c + 2 * i), 2 * i + 1 < V ? load_param<T>(p, a.wf32, c + 2 * i + 1) : 0.f);
  }
}

// sigmoid(z) and z sigmoid(z) of a pair; the latter closes at z = -inf (where
// the product would be 0 inf).
__device__ __forceinline__ void gate_of(uint64_t z, uint64_t& sg, uint64_t& act, bool sigmoid) {
  float a, b;
  unpack2(z, a, b);
  const float sa = sigmoid_f(a), sb = sigmoid_f(b);
  sg = pack2(sa, sb);
  act = sigmoid ? sg : pack2(a == -INFINITY ? 0.f : a * sa, b == -INFINITY ? 0.f : b * sb);
}
__device__ __forceinline__ uint64_t both(float a) { return pack2(a, a); }

}  // namespace gdr
