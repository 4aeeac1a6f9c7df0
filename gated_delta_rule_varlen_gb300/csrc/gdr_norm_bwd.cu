// gdr_norm_bwd.cu -- backward of the norms around a block (gdr_norm.cuh), and
// their entry points.  With hn = h r2 and xn = x r1:
//   dn = dy w,  dH = dh + r2 (dn - hn mean(dn hn)),  dw = sum_rows dy hn
//   dresidual = dH,  du = alpha dH
//   dz = du n act'(z)  (n = xn w_post or x),  du = du act(z)
//   dm = du w_post,  dx = r1 (dm - xn mean(dm xn)),  dw_post = sum_rows du xn
// A row of one element has no direction but its own, where the difference dn -
// hn mean(dn hn) is dn (1 - hn^2) = dn eps r2^2; it is formed that way, since the
// FP32 difference would keep nothing of it.
// The forward's values are formed again from the inputs, in FP32, so nothing
// is saved and no rounded h enters the gradients.
#include "gdr_norm.cuh"

namespace gdr {
namespace {

// Bound by HBM.  A block keeps its columns' weight gradients in registers over
// all its rows and leaves one partial row; k_norm_wgrad adds those.
template <typename T, int V, int TPR, int NV>
__global__ void __launch_bounds__(norm_threads(TPR)) k_norm_bwd(NormArgs a) {
  using G = RowGroup<TPR>;
  __shared__ float2 sm[3][G::WARPS];
  extern __shared__ float sred[];  // [GROUPS][D] when a block works on several rows
  const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const float inv_d = 1.f / (float)a.D;
  float dw[NV][V], dwp[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) dw[i][v] = dwp[i][v] = 0.f;
  for (int64_t base = (int64_t)blockIdx.x * G::GROUPS; base < a.rows; base += (int64_t)gridDim.x * G::GROUPS) {
    const int64_t r = base + grp;
    const bool live = r < a.rows;
    Vec<T, V> xr[NV], zr[NV], rr[NV], hr[NV], yr[NV];
    if (live) {
      const T* xp = row_ptr<T>(a.x, r, a.R1);
      const T* zp = a.gate.p ? row_ptr<T>(a.gate, r, a.R1) : nullptr;
      const T* rp = a.res.p ? row_ptr<T>(a.res, r, a.R1) : nullptr;
      const T* hp = a.dh.p ? row_ptr<T>(a.dh, r, a.R1) : nullptr;
      const T* yp = a.dy.p ? row_ptr<T>(a.dy, r, a.R1) : nullptr;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * V;
        if (c < a.D) {
          xr[i] = vload<T, V>(xp + c);
          if (zp) zr[i] = vload<T, V>(zp + c);
          if (rp) rr[i] = vload<T, V>(rp + c);
          if (hp) hr[i] = vload<T, V>(hp + c);
          if (yp) yr[i] = vload<T, V>(yp + c);
        }
      }
    }
    // r1
    float r1 = 1.f, s = 0.f, s2 = 0.f;
    if (a.w_post) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (live && (i * TPR + lane) * V < a.D) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float x = to_f<T>(xr[i].e[v]);
            s = fmaf(x, x, s);
          }
        }
      G::sum2(s, s2, sm[0]);
      r1 = rsqrtf(fmaf(s, inv_d, a.eps));
    }
    // h, its mean square and mean(dy w h)
    float h[NV][V];
    float r2 = 0.f, c2 = 0.f;
    s = 0.f;
    s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      const bool on = live && c < a.D;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[i][v] = 0.f;
        if (!on || !a.dy.p) continue;
        float u = to_f<T>(xr[i].e[v]);
        if (a.w_post) u *= r1 * load_param<T>(a.w_post, a.wf32, c + v);
        if (a.gate.p) {
          const float z = to_f<T>(zr[i].e[v]);
          u *= a.sigmoid ? sigmoid_f(z) : silu_f(z);
        }
        if (a.res.p) u = fmaf(a.alpha, u, to_f<T>(rr[i].e[v]));
        h[i][v] = u;
        s = fmaf(u, u, s);
        s2 = fmaf(to_f<T>(yr[i].e[v]) * load_param<T>(a.w, a.wf32, c + v), u, s2);
      }
    }
    if (a.dy.p) {
      G::sum2(s, s2, sm[1]);
      r2 = rsqrtf(fmaf(s, inv_d, a.eps));
      c2 = s2 * r2 * inv_d;  // mean(dn hn)
    }
    // dH, dresidual, dgate, du; mean(dm xn)
    s = 0.f;
    s2 = 0.f;
    float du[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      const bool on = live && c < a.D;
      float dH[V], dz[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        du[i][v] = 0.f;
        dH[v] = 0.f;
        dz[v] = 0.f;
        if (!on) continue;
        float g = a.dh.p ? to_f<T>(hr[i].e[v]) : 0.f;
        if (a.dy.p) {
          const float dy = to_f<T>(yr[i].e[v]), hn = h[i][v] * r2;
          dw[i][v] = fmaf(dy, hn, dw[i][v]);
          const float dn = dy * load_param<T>(a.w, a.wf32, c + v);
          g += r2 * (a.D > 1 ? dn - hn * c2 : dn * a.eps * r2 * r2);
        }
        dH[v] = g;
        g *= a.alpha;
        const float x = to_f<T>(xr[i].e[v]), wp = a.w_post ? load_param<T>(a.w_post, a.wf32, c + v) : 1.f;
        if (a.gate.p) {
          const float z = to_f<T>(zr[i].e[v]), sg = sigmoid_f(z);
          const float act = a.sigmoid ? sg : silu_f(z);
          const float dact = a.sigmoid ? sg * (1.f - sg) : fmaf(act, 1.f - sg, sg);
          dz[v] = g * (x * r1 * wp) * dact;
          g *= act;
        }
        if (a.w_post) {
          dwp[i][v] = fmaf(g, x * r1, dwp[i][v]);
          g *= wp;
          s = fmaf(g, x, s);
        }
        du[i][v] = g;
      }
      if (on) {
        if (a.dres) vstore<T, V>(static_cast<T*>(a.dres) + r * a.D + c, dH);
        if (a.dgate) vstore<T, V>(static_cast<T*>(a.dgate) + r * a.D + c, dz);
      }
    }
    if (a.w_post) {
      G::sum2(s, s2, sm[2]);
      const float c1 = s * r1 * inv_d;  // mean(dm xn)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float xn = live && (i * TPR + lane) * V < a.D ? to_f<T>(xr[i].e[v]) * r1 : 0.f;
          du[i][v] = r1 * (a.D > 1 ? du[i][v] - xn * c1 : du[i][v] * a.eps * r1 * r1);
        }
    }
    if (a.dx && live) {
      T* dxp = static_cast<T*>(a.dx) + r * a.D;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * V;
        if (c < a.D) vstore<T, V>(dxp + c, du[i]);
      }
    }
    // rows that run one sum only would meet its buffer again
    if (TPR > 32 && !a.w_post) __syncthreads();
  }
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.D;
  auto leave = [&](float (&g)[NV][V], float* to) {
    if constexpr (G::GROUPS == 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * V;
        if (c < a.D) {
#pragma unroll
          for (int v = 0; v < V; ++v) to[c + v] = g[i][v];
        }
      }
    } else {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * V;
        if (c < a.D) {
#pragma unroll
          for (int v = 0; v < V; ++v) sred[grp * a.D + c + v] = g[i][v];
        }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.D; c += G::THREADS) {
        float sum = 0.f;
        for (int j = 0; j < G::GROUPS; ++j) sum += sred[j * a.D + c];
        to[c] = sum;
      }
    }
  };
  if (a.w) leave(dw, part);
  if (a.w_post) leave(dwp, part + a.D);
}

// dw and dw_post: the blocks' partial rows added in a fixed order.
__global__ void __launch_bounds__(512) k_norm_wgrad(const float* __restrict__ part, int blocks, int D, float* dw,
                                                    float* dwp) {
  float* to = blockIdx.y == 0 ? dw : dwp;
  if (!to) return;
  __shared__ float s[16][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (c < D)
    for (int i = row; i < blocks; i += 16) sum += part[((int64_t)i * 2 + blockIdx.y) * D + c];
  s[row][lane] = sum;
  __syncthreads();
  if (row == 0 && c < D) {
#pragma unroll
    for (int i = 1; i < 16; ++i) sum += s[i][lane];
    to[c] = sum;
  }
}

template <typename T, int VT>
cudaError_t launch_t(const NormArgs& a, const NormShape& s, int blocks, cudaStream_t st) {
#define GDR_NORM_CASE(v, tpr, nv)                                                                       \
  if (s.V == v && s.TPR == tpr && s.NV == nv) {                                                         \
    const size_t sm = RowGroup<tpr>::GROUPS > 1 ? (size_t)RowGroup<tpr>::GROUPS * a.D * sizeof(float) : 0; \
    k_norm_bwd<T, v, tpr, nv><<<blocks, norm_threads(tpr), sm, st>>>(a);                                \
    return cudaGetLastError();                                                                          \
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

cudaError_t launch_norm_bwd(const NormArgs& a, int dtype, const NormShape& s, int blocks, cudaStream_t st) {
  switch (dtype) {
    case GDR_DTYPE_BF16: return launch_t<__nv_bfloat16, 8>(a, s, blocks, st);
    case GDR_DTYPE_F16: return launch_t<__half, 8>(a, s, blocks, st);
    default: return launch_t<float, 4>(a, s, blocks, st);
  }
}

namespace {

// Most blocks of a backward on rows of D elements (norm_blocks over the shapes
// that such rows take): the partial rows its workspace has to hold.
int max_norm_blocks(int D) { return D <= 1024 ? 152 * 8 : D <= 2048 ? 152 * 4 : 152 * 2; }

// Whether rows of D elements at these addresses and strides can be read in
// 16-byte pieces.
bool rows16(const RowTensor& t, int V) {
  return !t.p || (((uintptr_t)t.p & 15) == 0 && t.s0 % V == 0 && t.s1 % V == 0);
}

// The threads that hold a row: 16-byte pieces where all rows allow them, else
// single elements.
NormShape norm_shape(int D, int dtype, bool vec) {
  const int V = dtype == GDR_DTYPE_F32 ? 4 : 8;
  if (vec && D % V == 0) {
    const int n = D / V;
    if (n <= 8) return {V, 8, 1};
    if (n <= 16) return {V, 16, 1};
    if (n <= 32) return {V, 32, 1};
    if (n <= 128) return {V, 128, 1};
    if (n <= 256) return {V, 256, 1};
    if (n <= 512) return {V, 512, 1};
    if (n <= 1024) return {V, 512, 2};
    if (n <= 2048) return {V, 1024, 2};
    return {V, 1024, 4};
  }
  if (D <= 256) return {1, 32, 8};
  if (D <= 2048) return {1, 256, 8};
  return {1, 1024, 16};
}

int norm_blocks(int64_t rows, int TPR) {
  const int threads = norm_threads(TPR);
  const int64_t need = (rows + threads / TPR - 1) / (threads / TPR);
  const int64_t most = 152 * (1024 / threads);
  return (int)(need < most ? need : most);
}

gdr_status norm_check(int dtype, int wdtype, int64_t R0, int32_t R1, int32_t D, const void* x, const void* residual,
                      const void* post_weight, const void* weight, int act) {
  if (dtype < 0 || dtype > GDR_DTYPE_F32 || (wdtype != dtype && wdtype != GDR_DTYPE_F32)) return GDR_INVALID_ARG;
  if (R0 < 0 || R1 <= 0 || D <= 0 || D > GDR_NORM_MAX_D || (act != GDR_ACT_SILU && act != GDR_ACT_SIGMOID))
    return GDR_INVALID_ARG;
  if (R0 > 0 && !x) return GDR_INVALID_ARG;
  if (R0 > 0 && !residual && !post_weight && !weight) return GDR_INVALID_ARG;  // nothing to normalize or add
  return GDR_OK;
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

gdr_status norm_workspace_bytes(int32_t D, size_t* scratch_bytes) {
  if (!scratch_bytes || D <= 0 || D > GDR_NORM_MAX_D) return GDR_INVALID_ARG;
  *scratch_bytes = (size_t)max_norm_blocks(D) * 2 * D * sizeof(float);
  return GDR_OK;
}

gdr_status norm_fwd(int dtype, int64_t R0, int32_t R1, int32_t D, const void* x, int64_t xs0, int64_t xs1,
                    const void* gate, int64_t gs0, int64_t gs1, int act, const void* residual, int64_t rs0,
                    int64_t rs1, float res_scale, const void* post_weight, const void* weight, int wdtype, float eps,
                    void* h, void* y, cudaStream_t stream) {
  gdr_status rc = norm_check(dtype, wdtype, R0, R1, D, x, residual, post_weight, weight, act);
  if (rc != GDR_OK) return rc;
  if (R0 == 0) return GDR_OK;
  if ((!h && !y) || (y && !weight)) return GDR_INVALID_ARG;
  if ((rc = check_device()) != GDR_OK) return rc;
  NormArgs a{};
  a.rows = R0 * R1;
  a.R1 = R1;
  a.D = D;
  a.x = {x, xs0, xs1};
  a.gate = {gate, gs0, gs1};
  a.res = {residual, rs0, rs1};
  a.w_post = post_weight;
  a.w = weight;
  a.wf32 = wdtype == GDR_DTYPE_F32;
  a.sigmoid = act == GDR_ACT_SIGMOID;
  a.alpha = residual ? res_scale : 1.f;
  a.eps = eps;
  a.h = h;
  a.y = y;
  const int V = dtype == GDR_DTYPE_F32 ? 4 : 8;
  const bool vec = rows16(a.x, V) && rows16(a.gate, V) && rows16(a.res, V) &&
                   (((uintptr_t)h | (uintptr_t)y) & 15) == 0;
  const NormShape s = norm_shape(D, dtype, vec);
  ProfScope ps("norm_fwd", stream, (double)a.rows * D);
  return launch_norm_fwd(a, dtype, s, norm_blocks(a.rows, s.TPR), stream) == cudaSuccess ? GDR_OK : GDR_CUDA_ERROR;
}

gdr_status norm_bwd(int dtype, int64_t R0, int32_t R1, int32_t D, const void* x, int64_t xs0, int64_t xs1,
                    const void* gate, int64_t gs0, int64_t gs1, int act, const void* residual, int64_t rs0,
                    int64_t rs1, float res_scale, const void* post_weight, const void* weight, int wdtype, float eps,
                    const void* dh, int64_t dhs0, int64_t dhs1, const void* dy, int64_t dys0, int64_t dys1, void* dx,
                    void* dgate, void* dresidual, float* dweight, float* dpost_weight, void* scratch,
                    size_t scratch_bytes, cudaStream_t stream) {
  gdr_status rc = norm_check(dtype, wdtype, R0, R1, D, x, residual, post_weight, weight, act);
  if (rc != GDR_OK) return rc;
  if ((R0 > 0 && !dh && !dy) || (dy && !weight) || (dgate && !gate) || (dresidual && !residual) ||
      (dweight && !weight) || (dpost_weight && !post_weight))
    return GDR_INVALID_ARG;
  if (!scratch || ((uintptr_t)scratch & 255) != 0) return GDR_INVALID_ARG;
  size_t need = 0;
  norm_workspace_bytes(D, &need);
  if (scratch_bytes < need) return GDR_WORKSPACE_TOO_SMALL;
  if ((rc = check_device()) != GDR_OK) return rc;
  NormArgs a{};
  a.rows = R0 * R1;
  a.R1 = R1;
  a.D = D;
  a.x = {x, xs0, xs1};
  a.gate = {gate, gs0, gs1};
  a.res = {residual, rs0, rs1};
  a.w_post = post_weight;
  a.w = weight;
  a.wf32 = wdtype == GDR_DTYPE_F32;
  a.sigmoid = act == GDR_ACT_SIGMOID;
  a.alpha = residual ? res_scale : 1.f;
  a.eps = eps;
  a.dh = {dh, dhs0, dhs1};
  a.dy = {dy, dys0, dys1};
  a.dx = dx;
  a.dgate = dgate;
  a.dres = dresidual;
  a.part = static_cast<float*>(scratch);
  const int V = dtype == GDR_DTYPE_F32 ? 4 : 8;
  const bool vec = rows16(a.x, V) && rows16(a.gate, V) && rows16(a.res, V) && rows16(a.dh, V) && rows16(a.dy, V) &&
                   (((uintptr_t)dx | (uintptr_t)dgate | (uintptr_t)dresidual) & 15) == 0;
  const NormShape s = norm_shape(D, dtype, vec);
  const int blocks = norm_blocks(a.rows, s.TPR);
  if (blocks > 0) {
    ProfScope ps("norm_bwd", stream, (double)a.rows * D);
    if (launch_norm_bwd(a, dtype, s, blocks, stream) != cudaSuccess) return GDR_CUDA_ERROR;
  }
  if (dweight || dpost_weight) {
    ProfScope ps("norm_wgrad", stream);
    k_norm_wgrad<<<dim3((D + 31) / 32, 2), 512, 0, stream>>>(a.part, blocks, D, dweight, dpost_weight);
    if (cudaGetLastError() != cudaSuccess) return GDR_CUDA_ERROR;
  }
  return GDR_OK;
}

}  // extern "C"
