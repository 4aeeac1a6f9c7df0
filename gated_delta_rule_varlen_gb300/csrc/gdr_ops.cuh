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

__device__ __forceinline__ float sigmoid_f(float z) { return 1.f / (1.f + __expf(-z)); }
// z sigmoid(z): 0 for z = -inf, where the product would be 0 * inf.
__device__ __forceinline__ float silu_f(float z) {
  const float e = __expf(-z);
  return e == INFINITY ? 0.f : z / (1.f + e);
}

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
