// gdr_ops.cuh -- shared pieces of the operators around the recurrence: element
// types, 16-byte vector access, activations, document lookup.
#pragma once
#include "gdr_common.cuh"

namespace gdr {

template <>
__device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

// V elements of T as one aligned access, unpacked to FP32 and packed from it
// (one rounding to nearest).
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> vload(const T* p) {
  return *reinterpret_cast<const Vec<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void vunpack(const Vec<T, V>& v, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = to_f<T>(v.e[i]);
}
template <typename T, int V>
__device__ __forceinline__ void vstore(T* p, const float (&f)[V]) {
  Vec<T, V> v;
#pragma unroll
  for (int i = 0; i < V; ++i) v.e[i] = from_f<T>(f[i]);
  *reinterpret_cast<Vec<T, V>*>(p) = v;
}

// Pairs of FP32 operations as one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 1 / (1 + e^-z) from the approximate base-2 exponential and reciprocal (0 at -inf, 1
// at inf, and 0 below z = -87, where it is no normal number).  For activations T in
// FP32 the product with log2(e) carries its rounding error along (as the factor 1 +
// err ln 2): within 6e-7 relative over the whole range.  For types of 16 bits, whose rounding
// is 5e-4 and more, it does not: |z| 6e-8 beside 3e-7.
template <typename T>
__device__ __forceinline__ float sigmoid_f(float z) {
  const float e = z * -LOG2E;
  float y = ex2(e), r;
  if constexpr (sizeof(T) == 4) {
    const float err = fmaf(-1.92596299e-8f, z, fmaf(-z, LOG2E, -e));  // log2(e) - LOG2E
    y *= fmaf(fminf(err, 1.f), 0.69314718f, 1.f);  // (at infinities err is NaN and y 0 or infinite: any factor will do)
  }
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + y));
  return r;
}

// V elements as pairs (a single one: the pair's low half, beside zero).
template <int V>
constexpr int pairs_of = (V + 1) / 2;
template <typename T, int V>
__device__ __forceinline__ void to_pairs(const Vec<T, V>& v, uint64_t (&f)[pairs_of<V>]) {
  if constexpr (V == 1) {
    f[0] = pack2(to_f<T>(v.e[0]), 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f[i] = pack2(to_f<T>(v.e[2 * i]), to_f<T>(v.e[2 * i + 1]));
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_pairs(T* p, const uint64_t (&f)[pairs_of<V>]) {
  float o[V + 1];
#pragma unroll
  for (int i = 0; i < pairs_of<V>; ++i) unpack2(f[i], o[2 * i], o[2 * i + 1]);
  Vec<T, V> v;
#pragma unroll
  for (int i = 0; i < V; ++i) v.e[i] = from_f<T>(o[i]);
  *reinterpret_cast<Vec<T, V>*>(p) = v;
}
template <int V>
__device__ __forceinline__ void zero_pairs(uint64_t (&f)[pairs_of<V>]) {
#pragma unroll
  for (int i = 0; i < pairs_of<V>; ++i) f[i] = 0;
}
// The sum of a pair.
__device__ __forceinline__ float sum_of(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  return a + b;
}

// A launch whose blocks may start before the stream's previous kernel has ended, once
// all of that kernel's blocks have called next_may_start(): what it does before
// previous_ended() overlaps.  previous_ended() returns when the previous kernel has
// ended and its writes are visible.
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void previous_ended() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<A&&>(args)...);
}

// A ring of DEP vectors of V elements a thread in shared memory, filled by
// asynchronous copies: rows of a walk asked for DEP steps ahead without holding
// registers.  Each thread reads its own copies only, so that its own waits order
// them.  Every step of the walk takes one push (of nothing past the end).
template <typename T, int V, int DEP, int THREADS>
struct RowRing {
  using Item = Vec<T, V>;
  static_assert(sizeof(Item) == 4 || sizeof(Item) == 8 || sizeof(Item) == 16, "cp.async sizes");
  Item* base;  // [DEP][THREADS], at this thread's element
  __device__ __forceinline__ explicit RowRing(void* smem) : base(static_cast<Item*>(smem) + threadIdx.x) {}
  __device__ __forceinline__ void push(int slot, const T* src, bool live) {
    if (live) {
      const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(base + slot * THREADS));
      if constexpr (sizeof(Item) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(d), "l"(src) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(d), "l"(src), "n"((int)sizeof(Item))
                     : "memory");
    }
  }
  __device__ __forceinline__ Item at(int slot) const { return base[slot * THREADS]; }
};

// Parameter element (weights and biases come in the activations' type or FP32).
template <typename T>
__device__ __forceinline__ float load_param(const void* p, bool f32, int64_t i) {
  return f32 ? __ldg(static_cast<const float*>(p) + i) : to_f<T>(static_cast<const T*>(p)[i]);
}

// The first document that ends after token t (cu non-decreasing, cu[N] > t):
// the document that holds t.
__device__ __forceinline__ int doc_of(const int* __restrict__ cu, int N, int t) {
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid + 1) > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

}  // namespace gdr
