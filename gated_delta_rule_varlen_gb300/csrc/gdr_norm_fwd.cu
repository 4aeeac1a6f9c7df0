// gdr_norm_fwd.cu -- forward of the norms around a block (gdr_norm.cuh).
#include "gdr_norm.cuh"

namespace gdr {
namespace {

// Bound by HBM: each input read and each output written once.  Rows are dealt
// to the blocks in turn; rows past the end keep their threads in the barriers.
template <typename T, int V, int TPR, int NV>
__global__ void __launch_bounds__(norm_threads(TPR)) k_norm_fwd(NormArgs a) {
  using G = RowGroup<TPR>;
  __shared__ float2 sm[2][G::WARPS];
  const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const float inv_d = 1.f / (float)a.D;
  for (int64_t base = (int64_t)blockIdx.x * G::GROUPS; base < a.rows; base += (int64_t)gridDim.x * G::GROUPS) {
    const int64_t r = base + grp;
    const bool live = r < a.rows;
    Vec<T, V> xr[NV], zr[NV], rr[NV];
    if (live) {
      const T* xp = row_ptr<T>(a.x, r, a.R1);
      const T* zp = a.gate.p ? row_ptr<T>(a.gate, r, a.R1) : nullptr;
      const T* rp = a.res.p ? row_ptr<T>(a.res, r, a.R1) : nullptr;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * V;
        if (c < a.D) {
          xr[i] = vload<T, V>(xp + c);
          if (zp) zr[i] = vload<T, V>(zp + c);
          if (rp) rr[i] = vload<T, V>(rp + c);
        }
      }
    }
    float u[NV][V];
    float ss = 0.f, dummy = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool on = live && (i * TPR + lane) * V < a.D;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        u[i][v] = on ? to_f<T>(xr[i].e[v]) : 0.f;
        ss = fmaf(u[i][v], u[i][v], ss);
      }
    }
    if (a.w_post) {
      G::sum2(ss, dummy, sm[0]);
      const float r1 = rsqrtf(fmaf(ss, inv_d, a.eps));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * V;
        if (c < a.D) {
#pragma unroll
          for (int v = 0; v < V; ++v) u[i][v] *= r1 * load_param<T>(a.w_post, a.wf32, c + v);
        }
      }
    }
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool on = live && (i * TPR + lane) * V < a.D;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (a.gate.p && on) {
          const float z = to_f<T>(zr[i].e[v]);
          u[i][v] *= a.sigmoid ? sigmoid_f(z) : silu_f(z);
        }
        if (a.res.p && on) u[i][v] = fmaf(a.alpha, u[i][v], to_f<T>(rr[i].e[v]));
        ss = fmaf(u[i][v], u[i][v], ss);
      }
    }
    if (a.h && live) {
      T* hp = static_cast<T*>(a.h) + r * a.D;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * V;
        if (c < a.D) vstore<T, V>(hp + c, u[i]);
      }
    }
    if (a.y) {
      G::sum2(ss, dummy, sm[1]);
      const float r2 = rsqrtf(fmaf(ss, inv_d, a.eps));
      if (live) {
        T* yp = static_cast<T*>(a.y) + r * a.D;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (i * TPR + lane) * V;
          if (c < a.D) {
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] = u[i][v] * r2 * load_param<T>(a.w, a.wf32, c + v);
            vstore<T, V>(yp + c, y);
          }
        }
      }
    }
    // a row that runs only one of the two sums would meet its own buffer again
    if (TPR > 32 && !(a.w_post && a.y)) __syncthreads();
  }
}

template <typename T, int VT>
cudaError_t launch_t(const NormArgs& a, const NormShape& s, int blocks, cudaStream_t st) {
#define GDR_NORM_CASE(v, tpr, nv)                                             \
  if (s.V == v && s.TPR == tpr && s.NV == nv) {                               \
    k_norm_fwd<T, v, tpr, nv><<<blocks, norm_threads(tpr), 0, st>>>(a);       \
    return cudaGetLastError();                                                \
  }
  GDR_NORM_CASE(VT, 8, 1)
  GDR_NORM_CASE(VT, 16, 1)
  GDR_NORM_CASE(VT, 32, 1)
  GDR_NORM_CASE(VT, 128, 1)
  GDR_NORM_CASE(VT, 256, 1)
  GDR_NORM_CASE(VT, 512, 1)
  GDR_NORM_CASE(VT, 512, 2)
  GDR_NORM_CASE(VT, 1024, 2)
  GDR_NORM_CASE(VT, 1024, 4)
  GDR_NORM_CASE(1, 32, 8)
  GDR_NORM_CASE(1, 256, 8)
  GDR_NORM_CASE(1, 1024, 16)
#undef GDR_NORM_CASE
  return cudaErrorInvalidConfiguration;
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, int dtype, const NormShape& s, int blocks, cudaStream_t st) {
  switch (dtype) {
    case GDR_DTYPE_BF16: return launch_t<__nv_bfloat16, 8>(a, s, blocks, st);
    case GDR_DTYPE_F16: return launch_t<__half, 8>(a, s, blocks, st);
    default: return launch_t<float, 4>(a, s, blocks, st);
  }
}

}  // namespace gdr
