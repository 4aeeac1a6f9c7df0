// gdr_lnorm_fwd.cu -- forward of the layer norm in front of a block (gdr_lnorm.cuh).
#include "gdr_lnorm.cuh"

namespace gdr {
namespace {

// Bound by HBM: each input read and each output written once.  Fractions of the copy rate for
// 2^27 elements of BF16, with / without a residual: 128 columns 0.84 / 0.80, 2048 0.80 / 0.80,
// 4096 0.92 / 0.73, 8192 0.84 / 0.51, 16384 0.72 / 0.45 (the two sums of a row, one after the
// other), 1021 0.47 / 0.33 (rows shifted to 16-byte pieces); FP32 2048 0.83 / 0.85.  RES: with a residual; without
// one, rows are asked for twice as far ahead (gdr_norm.cuh).
template <typename T, int V, int TPR, int NV, bool CLUSTER, bool SHIFT, bool RES>
__global__ void __launch_bounds__(norm_threads(TPR)) k_lnorm_fwd(NormArgs a) {
  using W = RowWorker<T, V, TPR, NV, CLUSTER, SHIFT, RES ? 2 : 1>;
  constexpr int P = W::P;
  __shared__ float2 sm[2][RowGroup<TPR, CLUSTER>::SUMS];
  extern __shared__ __align__(16) unsigned char lnorm_smem[];
  W w(a, lnorm_smem);
  previous_ended();
  const float inv_d = 1.f / (float)a.D;
  typename W::Weight wk, bk;
  w.keep(wk, a.w);
  w.keep(bk, a.w_post);
  w.in.add(0, a.x);
  if constexpr (RES) w.in.add(1, a.res);
  if constexpr (W::AHEAD) {
#pragma unroll
    for (int i = 0; i < W::DEPTH; ++i) w.ask(i);
  }
  const uint64_t alpha = both(a.alpha);
  int slot = 0;
#pragma unroll 1
  for (int64_t r = w.g.first; r - w.g.grp < a.rows; r += w.g.step) {
    if constexpr (W::AHEAD) cp_async_wait<W::DEPTH - 1>();
    else w.ask(0);
    auto on = [&](int i) { return r < a.rows && w.col(i) < a.D; };
    uint64_t h[NV][P], s2 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      zero_pairs<V>(h[i]);
      if (on(i)) {
        w.get(slot, 0, i, h[i]);
        if constexpr (RES) {
          uint64_t f[P];
          w.get(slot, 1, i, f);
#pragma unroll
          for (int q = 0; q < P; ++q) h[i][q] = fma2(alpha, h[i][q], f[q]);
        }
#pragma unroll
        for (int q = 0; q < P; ++q) s2 = add2(s2, h[i][q]);
      }
    }
    w.put(a.h, r, h);
    if (a.y) {
      float s[1] = {sum_of(s2)};
      w.g.sum(s, sm[0]);
      const float mean = s[0] * inv_d;
      s2 = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (on(i)) {
          w.sub(h[i], i, mean);
#pragma unroll
          for (int q = 0; q < P; ++q) s2 = fma2(h[i][q], h[i][q], s2);
        }
      s[0] = sum_of(s2);
      w.g.sum(s, sm[1]);
      const uint64_t rr = both(rsqrtf(fmaf(s[0], inv_d, a.eps)));
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (on(i)) {
          uint64_t f[P], b[P];
          if (a.w) {
            w.weight(wk, i, f);
#pragma unroll
            for (int q = 0; q < P; ++q) f[q] = mul2(rr, f[q]);
          } else {
#pragma unroll
            for (int q = 0; q < P; ++q) f[q] = rr;
          }
          if (a.w_post) {
            w.weight(bk, i, b);
#pragma unroll
            for (int q = 0; q < P; ++q) h[i][q] = fma2(h[i][q], f[q], b[q]);
          } else {
#pragma unroll
            for (int q = 0; q < P; ++q) h[i][q] = mul2(h[i][q], f[q]);
          }
        }
      w.put(a.y, r, h);
    }
    if constexpr (W::AHEAD) {  // (what was read from the slot has been used)
      w.ask(slot);
      slot = slot == W::DEPTH - 1 ? 0 : slot + 1;
    }
  }
}

template <typename T>
struct Launch {
  const NormArgs& a;
  const NormShape& s;
  int* parts;
  cudaStream_t st;
  template <int V, int TPR, int NV, bool CLUSTER, bool SHIFT>
  cudaError_t run() const {
    return a.res.p ? go<V, TPR, NV, CLUSTER, SHIFT, true>() : go<V, TPR, NV, CLUSTER, SHIFT, false>();
  }
  template <int V, int TPR, int NV, bool CLUSTER, bool SHIFT, bool RES>
  cudaError_t go() const {
    static Held held;
    return norm_launch(k_lnorm_fwd<T, V, TPR, NV, CLUSTER, SHIFT, RES>, a, s,
                       RowWorker<T, V, TPR, NV, CLUSTER, SHIFT, RES ? 2 : 1>::BYTES, 32, held, parts, st, true);
  }
};

}  // namespace

cudaError_t launch_lnorm_fwd(const NormArgs& a, int dtype, const NormShape& s, cudaStream_t st) {
  int parts = 0;
  switch (dtype) {
    case GDR_DTYPE_BF16: return dispatch_lnorm<8>(s, Launch<__nv_bfloat16>{a, s, &parts, st});
    case GDR_DTYPE_F16: return dispatch_lnorm<8>(s, Launch<__half>{a, s, &parts, st});
    default: return dispatch_lnorm<4>(s, Launch<float>{a, s, &parts, st});
  }
}

}  // namespace gdr
