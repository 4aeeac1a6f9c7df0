// gdr_lnorm_bwd.cu -- backward of the layer norm in front of a block (gdr_lnorm.cuh), and
// its entry points.  With n = (h - mean) r and dn = dy w:
//   dH = dh + r (dn - mean(dn) - n mean(dn n)),  dw = sum_rows dy n,  db = sum_rows dy
//   dresidual = dH,  dx = alpha dH
// The forward's values are formed again from the inputs, in FP32: nothing is saved and no
// rounded h enters.  A row of two elements has n^2 = 1 - eps r^2 in both, where the FP32
// difference would keep nothing of dn - mean(dn) - n mean(dn n) = (dn - mean(dn)) eps r^2;
// it is formed that way.
#include "gdr_lnorm.cuh"

namespace gdr {
namespace {

// Blocks an SM holds at least (which bounds the registers).
constexpr int lnorm_bwd_min_blocks(int TPR, int elements) {
  if (TPR > 32) return TPR > 384 ? 1 : TPR > 128 ? 2 : TPR == 128 ? 3 : TPR == 96 ? 4 : 6;
  return elements <= 8 ? 5 : 3;
}

// Bound by HBM.  Fractions of the copy rate for 2^27 elements of BF16, with residual and dh /
// without: 128 columns 0.89 / 0.84, 2048 0.93 / 0.61, 4096 0.93 / 0.58, 8192 0.81 / 0.48, 16384
// 0.48 / 0.31, 1021 0.39 / 0.27; FP32 2048 0.89 / 0.80.  A block keeps its columns' weight gradients in registers over all its rows
// and leaves one partial row of each.  RES: with a residual or dh; without them, rows are
// asked for twice as far ahead.
template <typename T, int V, int TPR, int NV, bool CLUSTER, bool SHIFT, bool RES>
__global__ void __launch_bounds__(norm_threads(TPR), lnorm_bwd_min_blocks(TPR, V * NV)) k_lnorm_bwd(NormArgs a) {
  using W = RowWorker<T, V, TPR, NV, CLUSTER, SHIFT, RES ? 4 : 2>;
  constexpr int P = W::P;
  __shared__ float2 sm[2][RowGroup<TPR, CLUSTER>::SUMS];
  extern __shared__ __align__(16) unsigned char lnorm_smem[];
  W w(a, lnorm_smem);
  previous_ended();
  next_may_start();  // (the sum of the partial rows)
  const float inv_d = 1.f / (float)a.D;
  typename W::Weight wk;
  w.keep(wk, a.w);
  w.in.add(0, a.x);
  w.in.add(1, a.dy);
  if constexpr (RES) {
    if (a.res.p) w.in.add(2, a.res);
    if (a.dh.p) w.in.add(3, a.dh);
  }
  uint64_t dw[NV][P], db[NV][P];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    zero_pairs<V>(dw[i]);
    zero_pairs<V>(db[i]);
  }
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
    auto dn_of = [&](int i, uint64_t (&f)[P]) {  // dy w
      w.get(slot, 1, i, f);
      if (a.w) {
        uint64_t c[P];
        w.weight(wk, i, c);
#pragma unroll
        for (int q = 0; q < P; ++q) f[q] = mul2(f[q], c[q]);
      }
    };
    uint64_t h[NV][P], s2 = 0, t2 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      zero_pairs<V>(h[i]);
      if (on(i)) {
        uint64_t f[P];
        w.get(slot, 0, i, h[i]);
        if (RES && a.res.p) {
          w.get(slot, RES ? 2 : 0, i, f);
#pragma unroll
          for (int q = 0; q < P; ++q) h[i][q] = fma2(alpha, h[i][q], f[q]);
        }
        dn_of(i, f);
#pragma unroll
        for (int q = 0; q < P; ++q) {
          s2 = add2(s2, h[i][q]);
          t2 = add2(t2, f[q]);
        }
      }
    }
    float s[2] = {sum_of(s2), sum_of(t2)};
    w.g.sum(s, sm[0]);
    const float mean = s[0] * inv_d, mean_dn = s[1] * inv_d;
    s2 = t2 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (on(i)) {
        uint64_t f[P];
        w.sub(h[i], i, mean);
        dn_of(i, f);
#pragma unroll
        for (int q = 0; q < P; ++q) {
          s2 = fma2(h[i][q], h[i][q], s2);
          t2 = fma2(f[q], h[i][q], t2);
        }
      }
    s[0] = sum_of(s2);
    s[1] = sum_of(t2);
    w.g.sum(s, sm[1]);
    const float rs = rsqrtf(fmaf(s[0], inv_d, a.eps));
    // r (dn - mean(dn)) - r n mean(dn n); of two elements r eps r^2 (dn - mean(dn))
    const uint64_t rr = both(rs), pa = both(a.D == 2 ? rs * a.eps * rs * rs : rs),
                   pb = both(a.D == 2 ? 0.f : -rs * rs * rs * s[1] * inv_d);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (on(i)) {
        uint64_t f[P], y[P];
        w.get(slot, 1, i, y);
        dn_of(i, f);
        const uint64_t mdn = both(-mean_dn);
#pragma unroll
        for (int q = 0; q < P; ++q) {
          dw[i][q] = fma2(y[q], mul2(h[i][q], rr), dw[i][q]);
          db[i][q] = add2(db[i][q], y[q]);
          h[i][q] = fma2(pa, add2(f[q], mdn), mul2(pb, h[i][q]));
        }
        if (RES && a.dh.p) {
          w.get(slot, RES ? 3 : 0, i, f);
#pragma unroll
          for (int q = 0; q < P; ++q) h[i][q] = add2(h[i][q], f[q]);
        }
      }
    if (RES) w.put(a.dres, r, h);
    if (a.dx) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < P; ++q) h[i][q] = mul2(alpha, h[i][q]);
      w.put(a.dx, r, h);
    }
    if constexpr (W::AHEAD) {  // (what was read from the slot has been used)
      w.ask(slot);
      slot = slot == W::DEPTH - 1 ? 0 : slot + 1;
    }
  }
  if constexpr (W::AHEAD) cp_async_wait<0>();
  constexpr int GROUPS = RowGroup<TPR, CLUSTER>::GROUPS;
  float* part = a.part + (int64_t)(blockIdx.x / w.g.cluster) * 2 * a.D;
  auto leave = [&](const uint64_t (&sums)[NV][P], float* to) {
    float* at = to;
    if constexpr (GROUPS > 1) {  // the groups' rows meet in shared memory, [GROUPS][D]
      __syncthreads();
      at = reinterpret_cast<float*>(lnorm_smem) + w.g.grp * a.D;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = w.col(i);
      float f[V + 1];
#pragma unroll
      for (int q = 0; q < P; ++q) unpack2(sums[i][q], f[2 * q], f[2 * q + 1]);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (SHIFT ? c + v >= 0 && c + v < a.D : c < a.D) at[c + v] = f[v];
    }
    if constexpr (GROUPS > 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < a.D; c += W::THREADS) {
        float sum = 0.f;
        for (int j = 0; j < GROUPS; ++j) sum += reinterpret_cast<const float*>(lnorm_smem)[j * a.D + c];
        to[c] = sum;
      }
    }
  };
  leave(dw, part);
  leave(db, part + a.D);
}

template <typename T>
struct Launch {
  const NormArgs& a;
  const NormShape& s;
  int* parts;
  cudaStream_t st;
  template <int V, int TPR, int NV, bool CLUSTER, bool SHIFT>
  cudaError_t run() const {
    return a.res.p || a.dh.p ? go<V, TPR, NV, CLUSTER, SHIFT, true>() : go<V, TPR, NV, CLUSTER, SHIFT, false>();
  }
  template <int V, int TPR, int NV, bool CLUSTER, bool SHIFT, bool RES>
  cudaError_t go() const {
    static Held held;
    // (the groups' weight gradients meet in the same bytes: at most V NV columns a thread)
    const size_t smem = std::max((size_t)RowWorker<T, V, TPR, NV, CLUSTER, SHIFT, RES ? 4 : 2>::BYTES,
                                 TPR <= 32 ? 128 * V * NV * sizeof(float) : (size_t)0);
    return norm_launch(k_lnorm_bwd<T, V, TPR, NV, CLUSTER, SHIFT, RES>, a, s, smem, norm_bwd_blocks(a.D), held, parts, st, true);
  }
};

gdr_status lnorm_args(NormArgs& a, int dtype, int wdtype, int64_t R0, int32_t R1, int32_t D, const void* x, int64_t xs0,
                      int64_t xs1, const void* residual, int64_t rs0, int64_t rs1, float res_scale, const void* weight,
                      const void* bias, float eps) {
  if (dtype < 0 || dtype > GDR_DTYPE_F32 || (wdtype != dtype && wdtype != GDR_DTYPE_F32)) return GDR_INVALID_ARG;
  if (R0 < 0 || R1 <= 0 || D <= 0 || D > GDR_NORM_MAX_D || (R0 > 0 && !x)) return GDR_INVALID_ARG;
  a.rows = R0 * R1;
  a.R1 = R1;
  a.D = D;
  a.x = {x, xs0, xs1};
  a.res = {residual, rs0, rs1};
  a.w = weight;
  a.w_post = bias;
  a.wf32 = wdtype == GDR_DTYPE_F32;
  a.wvec = (((uintptr_t)bias | (uintptr_t)weight) & 15) == 0;
  a.alpha = residual ? res_scale : 1.f;
  a.eps = eps;
  return GDR_OK;
}

}  // namespace

cudaError_t launch_lnorm_bwd(const NormArgs& a, int dtype, const NormShape& s, int* parts, cudaStream_t st) {
  switch (dtype) {
    case GDR_DTYPE_BF16: return dispatch_lnorm<8>(s, Launch<__nv_bfloat16>{a, s, parts, st});
    case GDR_DTYPE_F16: return dispatch_lnorm<8>(s, Launch<__half>{a, s, parts, st});
    default: return dispatch_lnorm<4>(s, Launch<float>{a, s, parts, st});
  }
}

}  // namespace gdr

using namespace gdr;

extern "C" {

gdr_status lnorm_workspace_bytes(int32_t D, size_t* scratch_bytes) { return norm_workspace_bytes(D, scratch_bytes); }

gdr_status lnorm_fwd(int dtype, int64_t R0, int32_t R1, int32_t D, const void* x, int64_t xs0, int64_t xs1,
                     const void* residual, int64_t rs0, int64_t rs1, float res_scale, const void* weight,
                     const void* bias, int wdtype, float eps, void* h, void* y, cudaStream_t stream) {
  NormArgs a{};
  gdr_status rc = lnorm_args(a, dtype, wdtype, R0, R1, D, x, xs0, xs1, residual, rs0, rs1, res_scale, weight, bias, eps);
  if (rc != GDR_OK) return rc;
  if (R0 == 0) return GDR_OK;
  if (!y || y == h) return GDR_INVALID_ARG;
  if ((rc = check_device()) != GDR_OK) return rc;
  a.h = h;
  a.y = y;
  RowLayout l{R0, R1, D, dtype == GDR_DTYPE_F32 ? 4 : 8};
  for (const RowTensor& t : {a.x, a.res}) l.input(t);
  for (const void* p : {h, y}) l.output(p);
  ProfScope ps("lnorm_fwd", stream, (double)a.rows * D);
  return launch_lnorm_fwd(a, dtype, lnorm_shape(l), stream) == cudaSuccess ? GDR_OK : GDR_CUDA_ERROR;
}

gdr_status lnorm_bwd(int dtype, int64_t R0, int32_t R1, int32_t D, const void* x, int64_t xs0, int64_t xs1,
                     const void* residual, int64_t rs0, int64_t rs1, float res_scale, const void* weight, int wdtype,
                     float eps, const void* dh, int64_t dhs0, int64_t dhs1, const void* dy, int64_t dys0, int64_t dys1,
                     void* dx, void* dresidual, float* dweight, float* dbias, void* scratch, size_t scratch_bytes,
                     cudaStream_t stream) {
  NormArgs a{};
  gdr_status rc =
      lnorm_args(a, dtype, wdtype, R0, R1, D, x, xs0, xs1, residual, rs0, rs1, res_scale, weight, nullptr, eps);
  if (rc != GDR_OK) return rc;
  if ((R0 > 0 && !dy) || (dresidual && !residual)) return GDR_INVALID_ARG;
  if (R0 > 0 && dx && dx == dresidual && res_scale != 1.f) return GDR_INVALID_ARG;
  if (!scratch || ((uintptr_t)scratch & 255) != 0) return GDR_INVALID_ARG;
  size_t need = 0;
  norm_workspace_bytes(D, &need);
  if (scratch_bytes < need) return GDR_WORKSPACE_TOO_SMALL;
  if ((rc = check_device()) != GDR_OK) return rc;
  a.dh = {dh, dhs0, dhs1};
  a.dy = {dy, dys0, dys1};
  a.dx = dx;
  a.dres = dresidual;
  a.part = static_cast<float*>(scratch);
  RowLayout l{R0, R1, D, dtype == GDR_DTYPE_F32 ? 4 : 8};
  for (const RowTensor& t : {a.x, a.res, a.dh, a.dy}) l.input(t);
  for (const void* p : {dx, dresidual}) l.output(p);
  int parts = 0;
  if (a.rows > 0) {
    ProfScope ps("lnorm_bwd", stream, (double)a.rows * D);
    if (launch_lnorm_bwd(a, dtype, lnorm_shape(l), &parts, stream) != cudaSuccess) return GDR_CUDA_ERROR;
  }
  if (dweight || dbias) {
    ProfScope ps("lnorm_wgrad", stream);
    if (launch_norm_wgrad(a.part, parts, D, dweight, dbias, stream) != cudaSuccess) return GDR_CUDA_ERROR;
  }
  return GDR_OK;
}

}  // extern "C"
