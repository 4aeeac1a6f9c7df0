// gdr_lnorm.cuh -- layer norm in front of a block, with the scaled residual:
//   h = residual + alpha x   or  x
//   y = (h - mean) r w + b,  r = (mean (h - mean)^2 + eps)^(-1/2)
// on the rows and machinery of gdr_norm.cuh.  The mean is taken first and the squares of
// what is left of it then, so that a row far from zero keeps its variance.
// NormArgs: w_post holds the bias; gate, h's activation and dgate are not used.
#pragma once
#include "gdr_norm.cuh"

namespace gdr {

cudaError_t launch_lnorm_fwd(const NormArgs& a, int dtype, const NormShape& s, cudaStream_t st);
cudaError_t launch_lnorm_bwd(const NormArgs& a, int dtype, const NormShape& s, int* parts, cudaStream_t st);

// A thread's vectors of a row: K tensors of rows asked for ahead in shared memory where
// that pays (or in registers), the weights in registers where they fit.
template <typename T, int V, int TPR, int NV, bool CLUSTER, bool SHIFT, int K>
struct RowWorker {
  static constexpr int ITEMS = K * NV, THREADS = norm_threads(TPR);
  static constexpr int DEPTH = rows_ahead(THREADS, ITEMS * V * (int)sizeof(T));
  static constexpr bool AHEAD = V * sizeof(T) >= 4 && DEPTH >= 1;  // (no copies of two bytes)
  using Rows = RowsAhead<T, AHEAD ? V : 8, ITEMS, DEPTH, THREADS, !SHIFT>;
  static constexpr int BYTES = AHEAD ? Rows::BYTES : 0;
  static constexpr int P = pairs_of<V>;

  const NormArgs& a;
  RowGroup<TPR, CLUSTER> g;
  int m;  // a shifted row's vectors start m elements before it, on 16 bytes
  Rows ahead;
  Cursor<T, K> in;  // the next row to ask for
  Vec<T, V> raw[AHEAD ? 1 : K][AHEAD ? 1 : NV];

  __device__ __forceinline__ RowWorker(const NormArgs& args, void* smem)
      : a(args), m(SHIFT ? (int)(g.first % V) * (args.D % V) % V : 0), ahead(smem), in(g.first, g.step, args.R1) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      in.p[k] = nullptr;
      in.by[k] = in.wrap[k] = 0;
    }
  }
  __device__ __forceinline__ int col(int i) const { return (i * g.lanes + g.lane) * V - m; }
  __device__ __forceinline__ bool whole(int i) const { return !SHIFT || (col(i) >= 0 && col(i) + V <= a.D); }
  __device__ __forceinline__ void ask(int slot) {
    if (in.r < a.rows) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (in.p[k])
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int c = col(i);
            if (c < a.D) {
              if constexpr (AHEAD)
                ahead.ask(slot, k * NV + i, in.p[k] + c, SHIFT ? min(V, a.D - c) * (int)sizeof(T) : V * (int)sizeof(T));
              else
                raw[k][i] = vload<T, V>(in.p[k] + c);
            }
          }
    }
    if constexpr (AHEAD) cp_async_commit();
    in.next();
  }
  // Vector i of tensor k: zero outside the row.
  __device__ __forceinline__ void get(int slot, int k, int i, uint64_t (&f)[P]) const {
    if constexpr (AHEAD) to_pairs<T, V>(ahead.get(slot, k * NV + i), f);
    else to_pairs<T, V>(raw[k][i], f);
    if (SHIFT && !whole(i)) clip_pairs<V>(f, col(i), a.D);
  }
  __device__ __forceinline__ void put(void* to, int64_t r, const uint64_t (&f)[NV][P]) const {
    if (!to || r >= a.rows) return;
    T* p = static_cast<T*>(to) + r * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (col(i) < a.D) {
        if (whole(i)) store_pairs<T, V>(p + col(i), f[i]);
        else store_clipped<T, V>(p, col(i), a.D, f[i]);
      }
  }
  // f - by on a row's elements (what lies outside the row stays zero).
  __device__ __forceinline__ void sub(uint64_t (&f)[P], int i, float by) const {
    const uint64_t b = V == 1 ? pack2(-by, 0.f) : both(-by);
#pragma unroll
    for (int q = 0; q < P; ++q) f[q] = add2(f[q], b);
    if (SHIFT && !whole(i)) clip_pairs<V>(f, col(i), a.D);
  }
  // The weight's vectors in registers, but for blocks that leave a thread 64 of them.
  static constexpr bool KEEP = TPR < 1024;
  struct Weight {
    const void* p;
    uint64_t kept[KEEP ? NV : 1][P];
  };
  __device__ __forceinline__ void keep(Weight& w, const void* p) const {
    w.p = p;
    if constexpr (KEEP)
      if (p) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (col(i) < a.D) load_weight<T, V, SHIFT>(a, p, col(i), w.kept[i]);
      }
  }
  __device__ __forceinline__ void weight(const Weight& w, int i, uint64_t (&f)[P]) const {
    if constexpr (KEEP) {
#pragma unroll
      for (int q = 0; q < P; ++q) f[q] = w.kept[i][q];
    } else {
      load_weight<T, V, SHIFT>(a, w.p, col(i), f);
    }
  }
};

// The threads of a row: those of the other norms (norm_shape), but that wide rows of 16 bits
// have two pieces a thread: what a row costs beside its elements, the instructions of two
// sums, is shared by 16 of them.
inline NormShape lnorm_shape(const RowLayout& l) {
  const NormShape s = norm_shape(l);
  const int n = s.shift ? (l.D + 2 * l.V - 2) / l.V : l.D / l.V;
  if (s.V == 8 && n > 256)
    for (int tpr : {256, 384, 512, 768, 1024})
      if (n <= 2 * tpr) return {8, tpr, 2, 0, s.shift};
  return s;
}

// launch.run<V, TPR, NV, CLUSTER, SHIFT>() of a shape.
template <int VT, typename L>
cudaError_t dispatch_lnorm(const NormShape& s, L launch) {
#define GDR_LNORM_CASE(v, tpr, nv, cl, sh)                                                \
  if (s.V == v && s.TPR == tpr && s.NV == nv && (s.cluster > 0) == cl && s.shift == sh)   \
    return launch.template run<v, tpr, nv, cl, sh>();
#define GDR_LNORM_CASES(tpr, nv, cl)     \
  GDR_LNORM_CASE(VT, tpr, nv, cl, false) \
  GDR_LNORM_CASE(VT, tpr, nv, cl, true)
  GDR_LNORM_CASES(2, 1, false)
  GDR_LNORM_CASES(4, 1, false)
  GDR_LNORM_CASES(8, 1, false)
  GDR_LNORM_CASES(8, 2, false)
  GDR_LNORM_CASES(16, 2, false)
  GDR_LNORM_CASES(32, 2, false)
  GDR_LNORM_CASES(64, 2, false)
  GDR_LNORM_CASES(96, 2, false)
  GDR_LNORM_CASES(128, 2, false)
  GDR_LNORM_CASES(256, 2, false)
  GDR_LNORM_CASES(384, 2, false)
  GDR_LNORM_CASES(512, 2, false)
  if constexpr (VT == 4) {
    GDR_LNORM_CASES(640, 2, false)
  }
  GDR_LNORM_CASES(768, 2, false)
  GDR_LNORM_CASES(1024, 2, false)
  GDR_LNORM_CASES(128, 2, true)
  GDR_LNORM_CASE(1, 32, 8, false, false)
  GDR_LNORM_CASE(1, 128, 8, true, false)
#undef GDR_LNORM_CASES
#undef GDR_LNORM_CASE
  return cudaErrorInvalidConfiguration;
}

}  // namespace gdr
