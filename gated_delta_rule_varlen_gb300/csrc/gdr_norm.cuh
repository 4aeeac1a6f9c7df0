// gdr_norm.cuh -- the norms around a block, fused with its gate and residual:
//   u = x                          or  x r1 w_post,  r1 = (mean x^2 + eps)^(-1/2)
//   u = u act(z)                   with a gate z: act = silu or sigmoid
//   h = residual + alpha u         or  u
//   y = h r2 w,                    r2 = (mean h^2 + eps)^(-1/2)
// Every step is optional.  A row (of D elements) is held in registers from its
// one read to its one write, by a few lanes of a warp, by a block, or, past 2048
// elements of BF16, by a cluster of blocks; the means are FP32 sums by shuffles
// (and across warps and blocks through shared memory) in a fixed order.
#pragma once
#include "gdr_ops.cuh"
#include <algorithm>
#include <atomic>

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
  float* part;             // [row groups][2][D]: partial dw, dw_post
};

// The threads of a row, with NV vectors of V elements each: TPR <= 32 lanes (a block
// of 128 threads works on 128 / TPR rows at a time), a block of TPR threads, or
// `cluster` > 0 blocks of 128.  shift: rows of any length whose pieces of 16 bytes
// start before the row (norm_shape).
constexpr int MAX_CLUSTER = 16;
struct NormShape {
  int V, TPR, NV, cluster, shift;
};
constexpr int norm_threads(int TPR) { return TPR <= 32 ? 128 : TPR; }

cudaError_t launch_norm_fwd(const NormArgs& a, int dtype, const NormShape& s, cudaStream_t st);
// *parts: how many partial rows of weight gradients it left
cudaError_t launch_norm_bwd(const NormArgs& a, int dtype, const NormShape& s, int* parts, cudaStream_t st);

// Most blocks of an SM that a backward on rows of D elements is launched with.
constexpr int norm_bwd_blocks(int D) { return D <= 2048 ? 8 : 3; }

// What a device holds of a kernel at a time, kept from call to call (and from thread to
// thread): blocks an SM, or clusters by their size.  0: not known yet.
struct Held {
  static constexpr int DEVICES = 16;
  std::atomic<int> n[DEVICES][MAX_CLUSTER + 1];
};

// Launches as many row groups (blocks or clusters, each goes through its share of
// the rows) as the GPU holds at a time, `limit` blocks an SM at most, or fewer where
// there are fewer rows; a shifted row keeps its place within 16 bytes from one of a
// thread's rows to the next (the step between them is a multiple of V).  held: the
// kernel's own; smem is always the same for a kernel.
template <typename K>
cudaError_t norm_launch(K kernel, const NormArgs& a, const NormShape& s, size_t smem, int limit, Held& held, int* parts,
                        cudaStream_t st) {
  const int threads = norm_threads(s.TPR), groups = threads / s.TPR, size = s.cluster > 0 ? s.cluster : 1;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = size;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = s.cluster > 0 ? 1 : 0;
  // (a device's own setting, so not kept from call to call)
  if (smem > 40 << 10) {
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) return e;
  }
  if (s.cluster > 8) {
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) return e;
  }
  int dev = 0, fits = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  std::atomic<int>* known = dev >= 0 && dev < Held::DEVICES ? &held.n[dev][s.cluster] : nullptr;
  if (known) fits = known->load(std::memory_order_relaxed);
  if (fits == 0) {
    if (s.cluster > 0) {
      cfg.gridDim = dim3(152 / size * size);
      if (cudaError_t e = cudaOccupancyMaxActiveClusters(&fits, kernel, &cfg)) return e;
    } else if (cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fits, kernel, threads, smem)) {
      return e;
    }
    if (fits < 1) return cudaErrorInvalidConfiguration;
    if (known) known->store(fits, std::memory_order_relaxed);
  }
  // (the limit of this call's width, whatever width came first: the backward's workspace holds no more)
  const int most = s.cluster > 0 ? std::min(fits, 152 * limit / size) : 152 * std::min(fits, limit);
  int64_t n = std::min<int64_t>((a.rows + groups - 1) / groups, most);
  if (s.shift && s.V > groups) {
    const int64_t unit = s.V / groups;
    n = std::max(unit, n / unit * unit);
  }
  *parts = (int)n;
  cfg.gridDim = dim3((unsigned)(n * size));
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// v to the place of `at` in block `rank` of the cluster.
__device__ __forceinline__ void store_at_peer(float2* at, int rank, float2 v) {
  asm volatile(
      "{\n .reg .b32 p;\n mapa.shared::cluster.u32 p, %0, %1;\n st.shared::cluster.v2.f32 [p], {%2, %3};\n}\n" ::"r"(
          (uint32_t)__cvta_generic_to_shared(at)),
      "r"(rank), "f"(v.x), "f"(v.y)
      : "memory");
}

// This thread's place: its rows are first, first + step, ...; in each it has the
// vectors lane, lane + lanes, ...
template <int TPR, bool CLUSTER>
struct RowGroup {
  static constexpr int THREADS = norm_threads(TPR), GROUPS = THREADS / TPR;  // rows a block works on at a time
  static constexpr int WARPS = TPR > 32 ? TPR / 32 : 1, SUMS = CLUSTER ? WARPS * MAX_CLUSTER : WARPS;
  int lanes = TPR, lane = threadIdx.x % TPR, grp = threadIdx.x / TPR, rank = 0, cluster = 1;
  int64_t first = (int64_t)blockIdx.x * GROUPS + grp, step = (int64_t)gridDim.x * GROUPS;

  __device__ __forceinline__ RowGroup() {
    if constexpr (CLUSTER) {
      asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(rank));
      asm("mov.u32 %0, %%cluster_nctaid.x;\n" : "=r"(cluster));
      lanes = TPR * cluster;
      lane = TPR * rank + (int)threadIdx.x;
      first = blockIdx.x / cluster;
      step = gridDim.x / cluster;
      cluster_sync();  // the others' shared memory is there
    }
  }
  // All threads of the row.
  __device__ __forceinline__ void sync() const {
    if constexpr (CLUSTER) cluster_sync();
    else if constexpr (TPR > 32) __syncthreads();
  }
  // Sums of N values over the row's threads, on every thread of the row.  Two calls
  // in a row take different buffers: whoever writes one again has passed the
  // other's barrier, which its readers reach after it.
  template <int N>
  __device__ __forceinline__ void sum(float (&a)[N], float2* sm) const {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int m = W / 2; m >= 1; m >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) a[n] += __shfl_xor_sync(0xffffffffu, a[n], m);
    if constexpr (TPR > 32) {
      const int warp = threadIdx.x >> 5, in_warp = threadIdx.x & 31;
      const float2 own = make_float2(a[0], a[N - 1]);
      if constexpr (CLUSTER) {
        if (in_warp < cluster) store_at_peer(sm + rank * WARPS + warp, in_warp, own);
        cluster_sync();
      } else {
        if (in_warp == 0) sm[warp] = own;
        __syncthreads();
      }
#pragma unroll
      for (int n = 0; n < N; ++n) a[n] = 0.f;
      if constexpr (CLUSTER) {
#pragma unroll 1
        for (int i = 0; i < cluster; ++i) add<N>(a, sm + i * WARPS);
      } else {
        add<N>(a, sm);
      }
    }
  }

 private:
  template <int N>
  static __device__ __forceinline__ void add(float (&a)[N], const float2* sm) {
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
      const float2 v = sm[i];
      a[0] += v.x;
      if (N == 2) a[N - 1] += v.y;
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
// the thread a row, by asynchronous copies to shared memory, so that more bytes are
// in flight than registers would hold.  A thread reads its own copies only.  The
// threads' vectors lie side by side: with a thread's own together the gated norm's
// training took 1.4 times as long.
template <typename T, int V, int ITEMS, int DEPTH, int THREADS, bool WHOLE>
struct RowsAhead {
  using Item = Vec<T, V>;
  static constexpr int BYTES = ITEMS * DEPTH * THREADS * (int)sizeof(Item);
  Item* base;
  __device__ __forceinline__ explicit RowsAhead(void* smem) : base(static_cast<Item*>(smem) + threadIdx.x) {}
  // The first `bytes` of a vector, zeros behind (WHOLE: all).
  __device__ __forceinline__ void ask(int slot, int item, const T* src, int bytes) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(base + (slot * ITEMS + item) * THREADS));
    if constexpr (sizeof(Item) != 16)
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(d), "l"(src), "n"((int)sizeof(Item)) : "memory");
    else if constexpr (WHOLE)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(d), "l"(src) : "memory");
    else
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(d), "l"(src), "r"(bytes) : "memory");
  }
  __device__ __forceinline__ Item get(int slot, int item) const { return base[(slot * ITEMS + item) * THREADS]; }
};
// Rows ahead of kernels whose threads take `bytes` each a row: as many as fit what
// a block may take of shared memory, four at most.
constexpr int rows_ahead(int threads, int bytes) {
  const int room = threads <= 128 ? 40 << 10 : threads <= 256 ? 80 << 10 : threads <= 384 || (threads <= 512 && bytes <= 48) ? 100 << 10 : 200 << 10;
  const int n = room / (threads * bytes);
  return n < 4 ? n : 4;
}

// Vectors of a shifted row: elements before the row or past its end read as zero
// and are not written.
template <int V>
__device__ __forceinline__ void clip_pairs(uint64_t (&f)[pairs_of<V>], int c, int D) {
#pragma unroll
  for (int i = 0; i < pairs_of<V>; ++i) {
    float a, b;
    unpack2(f[i], a, b);
    const int k = c + 2 * i;
    f[i] = pack2(k >= 0 && k < D ? a : 0.f, k + 1 >= 0 && k + 1 < D ? b : 0.f);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_clipped(T* row, int c, int D, const uint64_t (&f)[pairs_of<V>]) {
#pragma unroll
  for (int i = 0; i < pairs_of<V>; ++i) {
    float a, b;
    unpack2(f[i], a, b);
    const int k = c + 2 * i;
    if (k >= 0 && k < D) row[k] = from_f<T>(a);
    if (k + 1 >= 0 && k + 1 < D) row[k + 1] = from_f<T>(b);
  }
}

// V elements of a weight from c on, in pairs.
template <typename T, int V, bool SHIFT>
__device__ __forceinline__ void load_weight(const NormArgs& a, const void* p, int c, uint64_t (&f)[pairs_of<V>]) {
  if constexpr (SHIFT) {
    auto at = [&](int k) { return k >= 0 && k < a.D ? load_param<T>(p, a.wf32, k) : 0.f; };
#pragma unroll
    for (int i = 0; i < pairs_of<V>; ++i) f[i] = pack2(at(c + 2 * i), at(c + 2 * i + 1));
  } else if (V > 1 && a.wvec) {
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
template <typename T>
__device__ __forceinline__ void gate_of(uint64_t z, uint64_t& sg, uint64_t& act, bool sigmoid) {
  float a, b;
  unpack2(z, a, b);
  const float sa = sigmoid_f<T>(a), sb = sigmoid_f<T>(b);
  sg = pack2(sa, sb);
  act = sigmoid ? sg : pack2(a == -INFINITY ? 0.f : a * sa, b == -INFINITY ? 0.f : b * sb);
}
__device__ __forceinline__ uint64_t both(float a) { return pack2(a, a); }

}  // namespace gdr
