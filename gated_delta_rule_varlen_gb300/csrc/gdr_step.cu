// gdr_step.cu -- one token of each sequence through the gated delta rule, the
// state updated in place:
//   S' = diag(exp g) S,  d = beta (v - S'^T k),  S = S' + k d^T,  out = scale S^T q
// with S^T q formed as S'^T q + (q . k) d, so that the state is read once,
// held in registers, and written once.
#include "gdr_ops.cuh"
#include "gdr_runtime.h"

namespace gdr {
namespace {

struct StepArgs {
  const __nv_bfloat16 *q, *k, *v;
  const float* g;
  const void* beta;
  float* state;      // [S][HV][128][128], S[k][v]
  const int* slots;  // [B] or null
  int B, S, Hqk, HV;
  float scale;
  int l2;
  __nv_bfloat16* out;
};

constexpr float kEps = 1e-6f;

// One block per (sequence, value head, 32 value columns): the columns of S do
// not meet in the update, so the slices are independent.  Thread (warp w, row
// group r, column quad c) holds rows w * 32 + 4 i + r of four columns.
// Bound by HBM: 128 KB of state a head.  128 sequences of 48 heads (805 MB) in 119-122 us,
// 98% of the copy rate.
template <bool VEC>  // VEC: per-channel gate and BF16 beta (KDA); else scalar gate and FP32 beta (GDN)
__global__ void __launch_bounds__(128) k_delta_step(StepArgs a) {
  __shared__ float sq[DK], sk[DK], sa[DK];
  __shared__ float4 red[2][4][8];
  const int j0 = (blockIdx.x & 3) * 32, h = (blockIdx.x >> 2) % a.HV, b = (blockIdx.x >> 2) / a.HV;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 3, c = lane & 7;
  const int slot = a.slots ? a.slots[b] : b;
  __nv_bfloat16* out = a.out + ((int64_t)b * a.HV + h) * DK + j0;
  if (slot < 0 || slot >= a.S) {  // an inactive row
    if (tid < 32) out[tid] = from_f<__nv_bfloat16>(0.f);
    return;
  }
  float4* S = reinterpret_cast<float4*>(a.state + ((int64_t)slot * a.HV + h) * DK * DK + j0) + c;
  float4 s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = S[(warp * 32 + 4 * i + r) * (DK / 4)];
  const int hq = h / (a.HV / a.Hqk);
  float q = to_f(a.q[((int64_t)b * a.Hqk + hq) * DK + tid]);
  float k = to_f(a.k[((int64_t)b * a.Hqk + hq) * DK + tid]);
  const float e = expf(VEC ? a.g[((int64_t)b * a.HV + h) * DK + tid] : a.g[(int64_t)b * a.HV + h]);
  // q.k and, for the in-kernel norm, |q|^2 and |k|^2
  float qk = q * k, qq = q * q, kk = k * k;
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) {
    qk += __shfl_xor_sync(0xffffffffu, qk, m);
    qq += __shfl_xor_sync(0xffffffffu, qq, m);
    kk += __shfl_xor_sync(0xffffffffu, kk, m);
  }
  __shared__ float3 dots[4];
  if (lane == 0) dots[warp] = make_float3(qk, qq, kk);
  sq[tid] = q;
  sk[tid] = k;
  sa[tid] = e;
  __syncthreads();
  qk = (dots[0].x + dots[1].x) + (dots[2].x + dots[3].x);
  float rq = 1.f, rk = 1.f;
  if (a.l2) {
    rq = rsqrtf((dots[0].y + dots[1].y) + (dots[2].y + dots[3].y) + kEps);
    rk = rsqrtf((dots[0].z + dots[1].z) + (dots[2].z + dots[3].z) + kEps);
    qk *= rq * rk;
  }
  float4 ks = make_float4(0.f, 0.f, 0.f, 0.f), qs = ks;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = warp * 32 + 4 * i + r;
    const float al = sa[n], kn = sk[n], qn = sq[n];
    s[i].x *= al; s[i].y *= al; s[i].z *= al; s[i].w *= al;
    ks.x = fmaf(kn, s[i].x, ks.x); ks.y = fmaf(kn, s[i].y, ks.y);
    ks.z = fmaf(kn, s[i].z, ks.z); ks.w = fmaf(kn, s[i].w, ks.w);
    qs.x = fmaf(qn, s[i].x, qs.x); qs.y = fmaf(qn, s[i].y, qs.y);
    qs.z = fmaf(qn, s[i].z, qs.z); qs.w = fmaf(qn, s[i].w, qs.w);
  }
#pragma unroll
  for (int m = 8; m <= 16; m <<= 1) {
    ks.x += __shfl_xor_sync(0xffffffffu, ks.x, m); ks.y += __shfl_xor_sync(0xffffffffu, ks.y, m);
    ks.z += __shfl_xor_sync(0xffffffffu, ks.z, m); ks.w += __shfl_xor_sync(0xffffffffu, ks.w, m);
    qs.x += __shfl_xor_sync(0xffffffffu, qs.x, m); qs.y += __shfl_xor_sync(0xffffffffu, qs.y, m);
    qs.z += __shfl_xor_sync(0xffffffffu, qs.z, m); qs.w += __shfl_xor_sync(0xffffffffu, qs.w, m);
  }
  if (r == 0) {
    red[0][warp][c] = ks;
    red[1][warp][c] = qs;
  }
  __syncthreads();
  const float beta = VEC ? to_f(static_cast<const __nv_bfloat16*>(a.beta)[(int64_t)b * a.HV + h])
                         : static_cast<const float*>(a.beta)[(int64_t)b * a.HV + h];
  const __nv_bfloat16* v = a.v + ((int64_t)b * a.HV + h) * DK + j0 + 4 * c;
  float d[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    auto col = [&](int m, int w) { return reinterpret_cast<const float*>(&red[m][w][c])[x]; };
    const float kS = rk * ((col(0, 0) + col(0, 1)) + (col(0, 2) + col(0, 3)));
    d[x] = beta * (to_f(v[x]) - kS);
    if (warp == 0 && r == 0) {
      const float qS = rq * ((col(1, 0) + col(1, 1)) + (col(1, 2) + col(1, 3)));
      out[4 * c + x] = from_f<__nv_bfloat16>(a.scale * fmaf(qk, d[x], qS));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = warp * 32 + 4 * i + r;
    const float kn = rk * sk[n];
    s[i].x = fmaf(kn, d[0], s[i].x);
    s[i].y = fmaf(kn, d[1], s[i].y);
    s[i].z = fmaf(kn, d[2], s[i].z);
    s[i].w = fmaf(kn, d[3], s[i].w);
    S[n * (DK / 4)] = s[i];
  }
}

gdr_status delta_step(bool vec, const void* q, const void* k, const void* v, const float* g, const void* beta,
                      float* state, const int32_t* slots, int32_t B, int32_t S, int32_t Hqk, int32_t HV, float scale,
                      int l2, void* out, cudaStream_t stream) {
  if (Hqk <= 0 || HV <= 0 || HV % Hqk != 0 || B < 0 || S < 0 || (!slots && B > S)) return GDR_INVALID_ARG;
  if (B == 0) return GDR_OK;
  if (!q || !k || !v || !g || !beta || !out || (S > 0 && !state)) return GDR_INVALID_ARG;
  if (((uintptr_t)state & 15) != 0 || (int64_t)B * HV * 4 > INT32_MAX) return GDR_INVALID_ARG;
  const gdr_status rc = check_device();
  if (rc != GDR_OK) return rc;
  StepArgs a{static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
             static_cast<const __nv_bfloat16*>(v), g, beta, state, slots, B, S, Hqk, HV, scale, l2,
             static_cast<__nv_bfloat16*>(out)};
  ProfScope ps(vec ? "kda_step" : "gdn_step", stream, (double)B * HV);
  if (vec) k_delta_step<true><<<B * HV * 4, 128, 0, stream>>>(a);
  else k_delta_step<false><<<B * HV * 4, 128, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? GDR_OK : GDR_CUDA_ERROR;
}

}  // namespace
}  // namespace gdr

extern "C" {

gdr_status kda_step(const gdr_bf16* q, const gdr_bf16* k, const gdr_bf16* v, const float* g, const gdr_bf16* beta,
                    float* state, const int32_t* slots, int32_t B, int32_t S, int32_t H, float scale, int qk_l2norm,
                    gdr_bf16* out, cudaStream_t stream) {
  return gdr::delta_step(true, q, k, v, g, beta, state, slots, B, S, H, H, scale, qk_l2norm, out, stream);
}

gdr_status gdn_step(const gdr_bf16* q, const gdr_bf16* k, const gdr_bf16* v, const float* g, const float* beta,
                    float* state, const int32_t* slots, int32_t B, int32_t S, int32_t Hqk, int32_t HV, float scale,
                    int qk_l2norm, gdr_bf16* out, cudaStream_t stream) {
  return gdr::delta_step(false, q, k, v, g, beta, state, slots, B, S, Hqk, HV, scale, qk_l2norm, out, stream);
}

}  // extern "C"
