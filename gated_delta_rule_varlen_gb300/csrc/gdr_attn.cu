// gdr_attn.cu -- softmax attention over packed documents: the entry points, and the
// kernels for shapes that the tensor cores' tiles do not take (gdr_attn.cuh has the
// formulas).
#include <cmath>

#include "gdr_attn_tc.cuh"

namespace gdr {
namespace {

constexpr int WARPS = 8;
constexpr int ME = GDR_ATTN_MAX_D / 32;  // elements of a row a lane holds

// A row's elements lane, lane + 32, ...
struct LaneRow {
  float e[ME];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int D) {
#pragma unroll
    for (int i = 0; i < ME; ++i) {
      const int d = (threadIdx.x & 31) + 32 * i;
      e[i] = d < D ? to_f(p[d]) : 0.f;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < ME; ++i) e[i] = 0.f;
  }
  __device__ __forceinline__ void add(float f, const LaneRow& x) {
#pragma unroll
    for (int i = 0; i < ME; ++i) e[i] = fmaf(f, x.e[i], e[i]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, int D, float f) const {
#pragma unroll
    for (int i = 0; i < ME; ++i) {
      const int d = (threadIdx.x & 31) + 32 * i;
      if (d < D) p[d] = from_f<__nv_bfloat16>(e[i] * f);
    }
  }
};
__device__ __forceinline__ float dot(const LaneRow& a, const LaneRow& b) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < ME; ++i) s = fmaf(a.e[i], b.e[i], s);
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  return s;
}

// One warp a query and head: one pass over its keys with the running maximum and sum.
// About 40 instructions a key and warp: the path for head dimensions and alignments
// that TMA does not address (32768 tokens of 16 heads of 128, causal: 1.33 s, on the tensor
// cores 2.9 ms).
__global__ void __launch_bounds__(WARPS * 32) k_attn_rows(AttnArgs a) {
  const int64_t item = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
  if (item >= a.T * a.H) return;
  const int t = (int)(item / a.H), h = (int)(item % a.H), hk = h / (a.H / a.HK);
  const int d = doc_of(a.cu, a.N, t), k0 = a.cuk[d];
  const KeyRange r = keys_of(a, t - a.cu[d], a.cu[d + 1] - a.cu[d], a.cuk[d + 1] - k0);
  const float c = a.scale * LOG2E;
  LaneRow q, acc, x;
  q.load(a.q.row(t, h), a.D);
  acc.zero();
  float m = -INFINITY, l = 0.f;
  for (int j = r.lo; j < r.hi; ++j) {
    x.load(a.k.row(k0 + j, hk), a.D);
    const float s = dot(q, x) * c;
    x.load(a.v.row(k0 + j, hk), a.D);
    const float top = fmaxf(m, s), base = top == -INFINITY ? 0.f : top;
    const float f = ex2(m - base), p = ex2(s - base);
    m = top;
    l = fmaf(l, f, p);
#pragma unroll
    for (int i = 0; i < ME; ++i) acc.e[i] = fmaf(acc.e[i], f, p * x.e[i]);
  }
  acc.store(a.out + item * a.D, a.D, l == 0.f ? 0.f : 1.f / l);
  if ((threadIdx.x & 31) == 0) a.lse[(int64_t)h * a.T + t] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
}

__device__ __forceinline__ float prob(float s, float c, float lse) { return lse == -INFINITY ? 0.f : ex2(fmaf(s, c, -lse * LOG2E)); }

// sum_j p (dp - delta) k_j as sum_j p dp k_j - delta sum_j p k_j: delta, the sum of p dp
// itself (over that of p, which is off 1 by lse's rounding), is known after the one pass.  (dout . out would bring the rounding of out along:
// where few keys are seen, 2^-8 of dp beside differences of dp.)
__global__ void __launch_bounds__(WARPS * 32) k_attn_dq_rows(AttnArgs a) {
  const int64_t item = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
  if (item >= a.T * a.H) return;
  const int t = (int)(item / a.H), h = (int)(item % a.H), hk = h / (a.H / a.HK);
  const int d = doc_of(a.cu, a.N, t), k0 = a.cuk[d];
  const KeyRange r = keys_of(a, t - a.cu[d], a.cu[d + 1] - a.cu[d], a.cuk[d + 1] - k0);
  const float c = a.scale * LOG2E, lse = a.lse_in[(int64_t)h * a.T + t];
  LaneRow q, g, k, v, pk, dk;
  q.load(a.q.row(t, h), a.D);
  g.load(a.dout.row(t, h), a.D);
  pk.zero();
  dk.zero();
  float delta = 0.f, all = 0.f;
  for (int j = r.lo; j < r.hi; ++j) {
    k.load(a.k.row(k0 + j, hk), a.D);
    v.load(a.v.row(k0 + j, hk), a.D);
    const float p = prob(dot(q, k), c, lse), pd = p * dot(g, v);
    delta += pd;
    all += p;
    pk.add(p, k);
    dk.add(pd, k);
  }
  if (all != 0.f) delta /= all;
  dk.add(-delta, pk);
  dk.store(a.dq + item * a.D, a.D, a.scale);
  if ((threadIdx.x & 31) == 0) a.delta[(int64_t)h * a.T + t] = delta;
}

// One warp a key and key head: all queries of its heads in their order.
__global__ void __launch_bounds__(WARPS * 32) k_attn_dkv_rows(AttnArgs a) {
  const int64_t item = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
  if (item >= a.TK * a.HK) return;
  const int t = (int)(item / a.HK), hk = (int)(item % a.HK), G = a.H / a.HK;
  const int d = doc_of(a.cuk, a.N, t), q0 = a.cu[d], lq = a.cu[d + 1] - q0, lk = a.cuk[d + 1] - a.cuk[d];
  const int j = t - a.cuk[d], at = j - (lk - lq);  // the query that j is the last key of
  const int lo = a.causal ? max(0, at) : 0, hi = a.window ? (int)min((int64_t)lq, (int64_t)at + a.window) : lq;
  const float c = a.scale * LOG2E;
  LaneRow k, v, dk, dv, q, g;
  k.load(a.k.row(t, hk), a.D);
  v.load(a.v.row(t, hk), a.D);
  dk.zero();
  dv.zero();
  for (int h = hk * G; h < (hk + 1) * G; ++h)
    for (int i = lo; i < hi; ++i) {
      q.load(a.q.row(q0 + i, h), a.D);
      g.load(a.dout.row(q0 + i, h), a.D);
      const int64_t s = h * a.T + q0 + i;
      const float p = prob(dot(q, k), c, a.lse_in[s]);
      dv.add(p, g);
      dk.add(p * (dot(g, v) - a.delta[s]), q);
    }
  dk.store(a.dk + item * a.D, a.D, a.scale);
  dv.store(a.dv + item * a.D, a.D, 1.f);
}

gdr_status attn_check(AttnArgs& a, const int32_t* cu_host, const int32_t* cuk_host) {
  int64_t nc = 0;
  gdr_status rc = plan_host(a.T, a.N, cu_host, &nc);
  if (rc != GDR_OK) return rc;
  if (a.cuk ? !cuk_host : cuk_host != nullptr) return GDR_INVALID_ARG;
  if (!cuk_host) {
    if (a.TK != a.T) return GDR_INVALID_ARG;
  } else if ((rc = plan_host(a.TK, a.N, cuk_host, &nc)) != GDR_OK) {
    return rc;
  }
  if (a.T > GDR_OPS_MAX_T || a.TK > GDR_OPS_MAX_T) return GDR_INVALID_ARG;
  if (a.H <= 0 || a.HK <= 0 || a.H % a.HK != 0 || a.D <= 0 || a.D > GDR_ATTN_MAX_D) return GDR_INVALID_ARG;
  if (a.window < 0 || (a.window > 0 && !a.causal)) return GDR_INVALID_ARG;
  if (!(a.scale > 0.f) || !std::isfinite(a.scale)) return GDR_INVALID_ARG;
  if ((a.T > 0 && !a.q.p) || (a.TK > 0 && (!a.k.p || !a.v.p))) return GDR_INVALID_ARG;
  if (a.N > 0 && !a.cu) return GDR_INVALID_ARG;
  for (int64_t rows : {a.T * a.H, a.TK * a.HK})  // (blocks of the kernels)
    if ((rows + WARPS - 1) / WARPS > INT32_MAX) return GDR_INVALID_ARG;
  if (!a.cuk) a.cuk = a.cu;
  return GDR_OK;
}

size_t delta_bytes(const AttnArgs& a) { return ((size_t)a.T * a.H * sizeof(float) + 255) / 256 * 256; }
unsigned blocks_of(int64_t rows) { return (unsigned)((rows + WARPS - 1) / WARPS); }

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

gdr_status attn_workspace_bytes(int64_t T, int64_t TK, int32_t H, int32_t HK, int32_t D, int32_t N,
                                const int32_t* cu_seqlens_host, const int32_t* cu_keys_host, int causal, int32_t window,
                                size_t* fwd_scratch_bytes, size_t* bwd_scratch_bytes) {
  AttnArgs a{};
  a.T = T;
  a.TK = TK;
  a.H = H;
  a.HK = HK;
  a.D = D;
  a.N = N;
  a.causal = causal != 0;
  a.window = window;
  a.scale = 1.f;
  a.q.p = a.k.p = a.v.p = reinterpret_cast<const __nv_bfloat16*>(16);  // (no pointers yet)
  a.cu = reinterpret_cast<const int*>(16);
  a.cuk = cu_keys_host ? a.cu : nullptr;
  if (const gdr_status rc = attn_check(a, cu_seqlens_host, cu_keys_host); rc != GDR_OK) return rc;
  AttnPlan p{};
  if (attn_tc_shape(D)) p = attn_plan(a, cu_seqlens_host, cu_keys_host ? cu_keys_host : cu_seqlens_host);
  if (fwd_scratch_bytes) *fwd_scratch_bytes = p.fwd_bytes;
  if (bwd_scratch_bytes) *bwd_scratch_bytes = delta_bytes(a) + p.bwd_bytes;
  return GDR_OK;
}

gdr_status attn_fwd(const gdr_bf16* q, int64_t qs0, int64_t qs1, const gdr_bf16* k, int64_t ks0, int64_t ks1,
                    const gdr_bf16* v, int64_t vs0, int64_t vs1, const int32_t* cu_seqlens,
                    const int32_t* cu_seqlens_host, const int32_t* cu_keys, const int32_t* cu_keys_host, int32_t N,
                    int64_t T, int64_t TK, int32_t H, int32_t HK, int32_t D, float scale, int causal, int32_t window,
                    gdr_bf16* out, float* lse, void* scratch, size_t scratch_bytes, cudaStream_t stream) {
  AttnArgs a{};
  a.q = {reinterpret_cast<const __nv_bfloat16*>(q), qs0, qs1};
  a.k = {reinterpret_cast<const __nv_bfloat16*>(k), ks0, ks1};
  a.v = {reinterpret_cast<const __nv_bfloat16*>(v), vs0, vs1};
  a.cu = cu_seqlens;
  a.cuk = cu_keys;
  a.N = N;
  a.T = T;
  a.TK = TK;
  a.H = H;
  a.HK = HK;
  a.D = D;
  a.scale = scale;
  a.causal = causal != 0;
  a.window = window;
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  gdr_status rc = attn_check(a, cu_seqlens_host, cu_keys_host);
  if (rc != GDR_OK) return rc;
  if (T == 0) return GDR_OK;
  if (!out || !lse || out == q || out == k || out == v) return GDR_INVALID_ARG;
  const bool tiles = attn_tc_shape(D) && attn_tc_layout(a);
  AttnPlan p{};
  const int32_t* keys_host = cu_keys_host ? cu_keys_host : cu_seqlens_host;
  if (tiles) {
    p = attn_plan(a, cu_seqlens_host, keys_host);
    if (p.fwd_bytes > 0 && (!scratch || ((uintptr_t)scratch & 255) != 0)) return GDR_INVALID_ARG;
    if (scratch_bytes < p.fwd_bytes) return GDR_WORKSPACE_TOO_SMALL;
  }
  if ((rc = check_device()) != GDR_OK) return rc;
  if (tiles)
    return launch_attn_fwd(a, p, cu_seqlens_host, keys_host, static_cast<float*>(scratch), stream) == cudaSuccess ? GDR_OK
                                                                                                                 : GDR_CUDA_ERROR;
  ProfScope ps("attn_rows", stream, (double)T * H);
  k_attn_rows<<<blocks_of(T * H), WARPS * 32, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? GDR_OK : GDR_CUDA_ERROR;
}

gdr_status attn_bwd(const gdr_bf16* q, int64_t qs0, int64_t qs1, const gdr_bf16* k, int64_t ks0, int64_t ks1,
                    const gdr_bf16* v, int64_t vs0, int64_t vs1, const gdr_bf16* out, const float* lse,
                    const gdr_bf16* dout, int64_t ds0, int64_t ds1, const int32_t* cu_seqlens,
                    const int32_t* cu_seqlens_host, const int32_t* cu_keys, const int32_t* cu_keys_host, int32_t N,
                    int64_t T, int64_t TK, int32_t H, int32_t HK, int32_t D, float scale, int causal, int32_t window,
                    gdr_bf16* dq, gdr_bf16* dk, gdr_bf16* dv, void* scratch, size_t scratch_bytes, cudaStream_t stream) {
  AttnArgs a{};
  a.q = {reinterpret_cast<const __nv_bfloat16*>(q), qs0, qs1};
  a.k = {reinterpret_cast<const __nv_bfloat16*>(k), ks0, ks1};
  a.v = {reinterpret_cast<const __nv_bfloat16*>(v), vs0, vs1};
  a.dout = {reinterpret_cast<const __nv_bfloat16*>(dout), ds0, ds1};
  a.cu = cu_seqlens;
  a.cuk = cu_keys;
  a.N = N;
  a.T = T;
  a.TK = TK;
  a.H = H;
  a.HK = HK;
  a.D = D;
  a.scale = scale;
  a.causal = causal != 0;
  a.window = window;
  a.o = reinterpret_cast<const __nv_bfloat16*>(out);
  a.lse_in = lse;
  a.dq = reinterpret_cast<__nv_bfloat16*>(dq);
  a.dk = reinterpret_cast<__nv_bfloat16*>(dk);
  a.dv = reinterpret_cast<__nv_bfloat16*>(dv);
  gdr_status rc = attn_check(a, cu_seqlens_host, cu_keys_host);
  if (rc != GDR_OK) return rc;
  if (T > 0 && (!dout || !out || !lse || !dq)) return GDR_INVALID_ARG;
  if (TK > 0 && (!dk || !dv)) return GDR_INVALID_ARG;
  for (const void* g : {(const void*)dq, (const void*)dk, (const void*)dv})
    for (const void* x : {(const void*)q, (const void*)k, (const void*)v, (const void*)out, (const void*)dout})
      if (g && g == x) return GDR_INVALID_ARG;
  if ((dq && (dq == dk || dq == dv)) || (dk && dk == dv)) return GDR_INVALID_ARG;
  if (T == 0 && TK == 0) return GDR_OK;
  const int32_t* keys_host = cu_keys_host ? cu_keys_host : cu_seqlens_host;
  AttnPlan p{};
  if (attn_tc_shape(D)) p = attn_plan(a, cu_seqlens_host, keys_host);
  const size_t need = delta_bytes(a) + p.bwd_bytes;
  if (need > 0 && (!scratch || ((uintptr_t)scratch & 255) != 0)) return GDR_INVALID_ARG;
  if (scratch_bytes < need) return GDR_WORKSPACE_TOO_SMALL;
  if ((rc = check_device()) != GDR_OK) return rc;
  a.delta = static_cast<float*>(scratch);
  if (attn_tc_shape(D) && attn_tc_layout(a)) {
    float* rest = reinterpret_cast<float*>(static_cast<char*>(scratch) + delta_bytes(a));
    return launch_attn_bwd(a, p, cu_seqlens_host, keys_host, rest, stream) == cudaSuccess ? GDR_OK : GDR_CUDA_ERROR;
  }
  if (T > 0) {
    ProfScope ps("attn_dq_rows", stream, (double)T * H);
    k_attn_dq_rows<<<blocks_of(T * H), WARPS * 32, 0, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return GDR_CUDA_ERROR;
  }
  if (TK > 0) {
    ProfScope ps("attn_dkv_rows", stream, (double)TK * HK);
    k_attn_dkv_rows<<<blocks_of(TK * HK), WARPS * 32, 0, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return GDR_CUDA_ERROR;
  }
  return GDR_OK;
}

}  // extern "C"
