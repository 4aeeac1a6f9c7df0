// gdr_ssm.cu -- the selective state space scan with a scalar decay a head, for
// packed prompts and for single tokens.  Per (document, head), state S [N][P]:
//   dt' = softplus(dt + dt_bias) (or dt + dt_bias),  S_t = exp(dt' A) S_{t-1} + dt' B_t x_t^T,
//   out_t = S_t^T C_t + D x_t
// head h reads B and C of group h / (H / G).
#include "gdr_ssm.cuh"

namespace gdr {
namespace {

// Token by token, for shapes and layouts that the chunked kernels do not take
// (state sizes above 128, sizes or rows that TMA cannot address) and for packs of
// short documents (short_documents()): one block per
// (document, head, 32 columns of the state), a warp four of them with the state's
// rows on its lanes, R a lane in registers; tokens staged through shared memory in
// tiles of 32 and taken four at a time, so that their sums over the lanes overlap.
// Bound by the chain of tokens: 0.19 us each up to 32 state rows, 0.30 us at 256.
constexpr int kSeqTok = 32;
template <int R>
__global__ void __launch_bounds__(256) k_ssm_seq(SsmArgs a) {
  __shared__ __align__(16) float sx[kSeqTok][32], sy[kSeqTok][32];
  __shared__ float sdt[kSeqTok], sda[kSeqTok];
  __shared__ __nv_bfloat16 sb[kSeqTok][32 * R], sc[kSeqTok][32 * R];
  const int slices = (a.P + 31) / 32;
  const int p0 = (blockIdx.x % slices) * 32, h = (blockIdx.x / slices) % a.H, d = blockIdx.x / slices / a.H;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = h / (a.H / a.G);
  const int t0 = a.cu[d], t1 = a.cu[d + 1], pw = p0 + 4 * warp;  // the warp's first column
  float s[R][4];
  const int64_t state = (((int64_t)d * a.H + h) * a.NS + lane) * a.P + pw;
  const bool quads = a.P % 4 == 0 && (((uintptr_t)a.h0 | (uintptr_t)a.ht) & 15) == 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float* from = a.h0 && lane + 32 * i < a.NS ? a.h0 + state + (int64_t)32 * i * a.P : nullptr;
    if (quads) {
      const float4 v = from && pw < a.P ? *reinterpret_cast<const float4*>(from) : make_float4(0.f, 0.f, 0.f, 0.f);
      s[i][0] = v.x, s[i][1] = v.y, s[i][2] = v.z, s[i][3] = v.w;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) s[i][q] = from && pw + q < a.P ? from[q] : 0.f;
    }
  }
  auto token = [&](int j) {
    const float4 x = *reinterpret_cast<const float4*>(&sx[j][4 * warp]);
    const float dt = sdt[j], da = sda[j], xd[4] = {x.x * dt, x.y * dt, x.z * dt, x.w * dt};
    float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float b = to_f(sb[j][lane + 32 * i]), c = to_f(sc[j][lane + 32 * i]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        s[i][q] = fmaf(da, s[i][q], b * xd[q]);
        y[q] = fmaf(c, s[i][q], y[q]);
      }
    }
    // the four sums over the lanes: halves of the warp take two each, quarters one
    const bool up = lane & 16, up2 = lane & 8;
    const float u = (up ? y[2] : y[0]) + __shfl_xor_sync(0xffffffffu, up ? y[0] : y[2], 16);
    const float v = (up ? y[3] : y[1]) + __shfl_xor_sync(0xffffffffu, up ? y[1] : y[3], 16);
    float w = (up2 ? v : u) + __shfl_xor_sync(0xffffffffu, up2 ? u : v, 8);
#pragma unroll
    for (int m = 4; m >= 1; m >>= 1) w += __shfl_xor_sync(0xffffffffu, w, m);
    if ((lane & 7) == 0) sy[j][4 * warp + (lane >> 3)] = w;
  };
  for (int t = t0; t < t1; t += kSeqTok) {
    const int len = min(kSeqTok, t1 - t);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSeqTok / 8; ++i) {
      const int j = warp + 8 * i;
      sx[j][lane] = j < len && p0 + lane < a.P ? to_f(a.x[(int64_t)(t + j) * a.ldx + h * a.P + p0 + lane]) : 0.f;
    }
    // (state rows past NS stay zero: B and C are zeros there)
#pragma unroll
    for (int i = 0; i < kSeqTok / 8; ++i) {
      const int j = warp + 8 * i;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int n = lane + 32 * r;
        const bool in = j < len && n < a.NS;
        sb[j][n] = in ? a.B[(int64_t)(t + j) * a.ldb + grp * a.NS + n] : __ushort_as_bfloat16(0);
        sc[j][n] = in ? a.C[(int64_t)(t + j) * a.ldc + grp * a.NS + n] : __ushort_as_bfloat16(0);
      }
    }
    if (threadIdx.x < len) {
      const float dt = load_dt(a, t + threadIdx.x, h);
      sdt[threadIdx.x] = dt;
      sda[threadIdx.x] = expf(dt * a.A[h]);
    }
    __syncthreads();
    int j = 0;
#pragma unroll 1
    for (; j + 4 <= len; j += 4) {
#pragma unroll
      for (int k = 0; k < 4; ++k) token(j + k);
    }
#pragma unroll 1
    for (; j < len; ++j) token(j);
    __syncthreads();
    for (int i = threadIdx.x; i < len * 32; i += 256) {
      const int j = i >> 5, l = i & 31;
      if (p0 + l < a.P)
        a.out[((int64_t)(t + j) * a.H + h) * a.P + p0 + l] =
            from_f<__nv_bfloat16>(fmaf(a.D ? a.D[h] : 0.f, sx[j][l], sy[j][l]));
    }
  }
  if (a.ht) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (lane + 32 * i >= a.NS) break;
      float* to = a.ht + state + (int64_t)32 * i * a.P;
      if (quads && pw < a.P) {
        *reinterpret_cast<float4*>(to) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (pw + q < a.P) to[q] = s[i][q];
      }
    }
  }
}

// One token of each sequence: one block per (sequence, head), each state row
// read, updated, multiplied by C and written in one pass.  256 threads cover
// P / V columns times the rows; the rows' partial sums meet in shared memory.
// Bound by HBM: 8 bytes a state element.  256 sequences of 64 heads x 128 x 64 (1.08 GB) in
// 157 us, the copy rate (200 us with B, C and dt awaited before the state is asked
// for).  V: four columns a thread where P and the pool's address allow it.
template <int V>
__global__ void __launch_bounds__(256) k_ssm_step(SsmArgs a) {
  __shared__ float sb[GDR_SSM_MAX_N], sc[GDR_SSM_MAX_N];
  __shared__ float red[256 * V];
  const int h = blockIdx.x % a.H, b = blockIdx.x / a.H, grp = h / (a.H / a.G);
  const int cols = (a.P + V - 1) / V, rows = 256 / cols;  // column groups, rows at a time
  const int c = threadIdx.x % cols, r = threadIdx.x / cols;
  const int slot = a.slots ? a.slots[b] : b;
  __nv_bfloat16* out = a.out + ((int64_t)b * a.H + h) * a.P;
  if (slot < 0 || slot >= a.S) {  // an inactive row
    for (int p = threadIdx.x; p < a.P; p += 256) out[p] = from_f<__nv_bfloat16>(0.f);
    return;
  }
  float* S = a.state + ((int64_t)slot * a.H + h) * a.NS * a.P + c * V;
  constexpr int U = 8;  // rows in flight a thread
  const int n_end = r < rows ? a.NS : 0;
  Vec<float, V> s[U];
  auto load = [&](int n0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (n0 + u * rows < n_end) s[u] = vload<float, V>(S + (int64_t)(n0 + u * rows) * a.P);
  };
  load(r);  // the state first: everything else is on its way meanwhile
  for (int n = threadIdx.x; n < a.NS; n += 256) {
    sb[n] = to_f(a.B[(int64_t)b * a.ldb + grp * a.NS + n]);
    sc[n] = to_f(a.C[(int64_t)b * a.ldc + grp * a.NS + n]);
  }
  const float dt = load_dt(a, b, h), da = expf(dt * a.A[h]);
  float xd[V], y[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    xd[v] = to_f(a.x[(int64_t)b * a.ldx + h * a.P + c * V + v]) * dt;
    y[v] = 0.f;
  }
  __syncthreads();
#pragma unroll 1
  for (int n0 = r; n0 < n_end; n0 += U * rows) {
    if (n0 != r) load(n0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = n0 + u * rows;
      if (n < n_end) {
        const float bn = sb[n], cn = sc[n];
        float t[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          t[v] = fmaf(da, s[u].e[v], bn * xd[v]);
          y[v] = fmaf(cn, t[v], y[v]);
        }
        vstore<float, V>(S + (int64_t)n * a.P, t);
      }
    }
  }
  if (r < rows) {
#pragma unroll
    for (int v = 0; v < V; ++v) red[(r * cols + c) * V + v] = y[v];
  }
  __syncthreads();
  for (int p = threadIdx.x; p < a.P; p += 256) {
    float sum = 0.f;
    for (int i = 0; i < rows; ++i) sum += red[i * cols * V + p];
    const float x = to_f(a.x[(int64_t)b * a.ldx + h * a.P + p]);
    out[p] = from_f<__nv_bfloat16>(fmaf(a.D ? a.D[h] : 0.f, x, sum));
  }
}

// Whether the documents are short enough to go token by token.  The chunked
// kernels work on 128 tokens whatever a document has; documents of up to 32 tokens
// (a tile) each are faster one by one, or nearly as fast at the end of that range: 64 of
// 64 heads x 128 x 64 states, with h0 and ht, take 109, 189, 281, 398 us at 2, 16, 32, 48
// tokens, in chunks 238-242; of 8 heads x 64 x 64 17, 25, 36, 48 against 36; of 32 heads x
// 32 x 128 46, 91, 148, 212 against 175-187.
bool short_documents(int N, const int32_t* cu) {
  for (int i = 0; i < N; ++i)
    if (cu[i + 1] - cu[i] > kSeqTok) return false;
  return true;
}

gdr_status ssm_check(const SsmArgs& a, int64_t T) {
  if (a.H <= 0 || a.G <= 0 || a.H % a.G != 0 || a.P <= 0 || a.P > GDR_SSM_MAX_P || a.NS <= 0 ||
      a.NS > GDR_SSM_MAX_N || T < 0)
    return GDR_INVALID_ARG;
  // a tile's end and a token's elements stay ints
  if (T > GDR_OPS_MAX_T || (int64_t)a.H * a.P > INT32_MAX || (int64_t)a.G * a.NS > INT32_MAX) return GDR_INVALID_ARG;
  if (T > 0 && (!a.x || !a.dt || !a.A || !a.B || !a.C || !a.out)) return GDR_INVALID_ARG;
  if (T > 1 && (a.ldx < (int64_t)a.H * a.P || a.ldb < (int64_t)a.G * a.NS || a.ldc < (int64_t)a.G * a.NS ||
                a.lddt < a.H))
    return GDR_INVALID_ARG;
  return GDR_OK;
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

gdr_status ssm_workspace_bytes(int64_t T, int32_t H, int32_t P, int32_t G, int32_t NS, int32_t N,
                               const int32_t* cu_seqlens_host, size_t* scratch_bytes) {
  int64_t nc = 0;
  if (T > GDR_OPS_MAX_T) return GDR_INVALID_ARG;
  if (!scratch_bytes || H <= 0 || G <= 0 || H % G != 0 || P <= 0 || P > GDR_SSM_MAX_P || NS <= 0 ||
      NS > GDR_SSM_MAX_N)
    return GDR_INVALID_ARG;
  const gdr_status rc = plan_host(T, N, cu_seqlens_host, &nc);
  if (rc != GDR_OK) return rc;
  *scratch_bytes = N > 0 && ssm_tc_shape(P, NS) ? ssm_tc_plan(H, P, NS, G, N, cu_seqlens_host).scratch : 0;
  return GDR_OK;
}

gdr_status ssm_fwd(const gdr_bf16* x, int64_t ldx, const void* dt, int dt_dtype, int64_t lddt, const float* A,
                   const gdr_bf16* B, int64_t ldb, const gdr_bf16* C, int64_t ldc, const float* D,
                   const float* dt_bias, int softplus, const int32_t* cu_seqlens, const int32_t* cu_seqlens_host,
                   int32_t N, int64_t T, int32_t H, int32_t P, int32_t G, int32_t NS, const float* h0, gdr_bf16* out,
                   float* ht, void* scratch, size_t scratch_bytes, cudaStream_t stream) {
  int64_t nc = 0;
  gdr_status rc = plan_host(T, N, cu_seqlens_host, &nc);
  if (rc != GDR_OK) return rc;
  if (dt_dtype != GDR_DTYPE_BF16 && dt_dtype != GDR_DTYPE_F32) return GDR_INVALID_ARG;
  SsmArgs a{};
  a.x = reinterpret_cast<const __nv_bfloat16*>(x);
  a.ldx = ldx;
  a.dt = dt;
  a.dt_f32 = dt_dtype == GDR_DTYPE_F32;
  a.lddt = lddt;
  a.A = A;
  a.B = reinterpret_cast<const __nv_bfloat16*>(B);
  a.C = reinterpret_cast<const __nv_bfloat16*>(C);
  a.ldb = ldb;
  a.ldc = ldc;
  a.D = D;
  a.dt_bias = dt_bias;
  a.softplus = softplus;
  a.cu = cu_seqlens;
  a.N = N;
  a.T = (int)T;
  a.H = H;
  a.P = P;
  a.G = G;
  a.NS = NS;
  a.h0 = h0;
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.ht = ht;
  if ((rc = ssm_check(a, T)) != GDR_OK) return rc;
  if (N == 0) return GDR_OK;
  if (!cu_seqlens) return GDR_INVALID_ARG;
  // The chunked kernels need rows that TMA can address; others go token by token.
  if (ssm_tc_shape(P, NS) && ssm_tc_layout(a)) {
    const SsmPlan plan = ssm_tc_plan(H, P, NS, G, N, cu_seqlens_host);
    if (plan.nseg * H * ((P + 63) / 64) > INT32_MAX) return GDR_INVALID_ARG;
    if (plan.scratch > 0 && (!scratch || ((uintptr_t)scratch & 255) != 0)) return GDR_INVALID_ARG;
    if (scratch_bytes < plan.scratch) return GDR_WORKSPACE_TOO_SMALL;
    if ((rc = check_device()) != GDR_OK) return rc;
    if (!short_documents(N, cu_seqlens_host))
      return launch_ssm_tc(a, plan, scratch, stream) == cudaSuccess ? GDR_OK : GDR_CUDA_ERROR;
  }
  const int64_t grid = (int64_t)N * H * ((P + 31) / 32);
  if (grid > INT32_MAX) return GDR_INVALID_ARG;
  if ((rc = check_device()) != GDR_OK) return rc;
  ProfScope ps("ssm_seq", stream, (double)T * H);
  static_assert(GDR_SSM_MAX_N <= 256, "eight state rows a lane");
  auto* kernel = NS <= 32 ? k_ssm_seq<1> : NS <= 64 ? k_ssm_seq<2> : NS <= 128 ? k_ssm_seq<4> : k_ssm_seq<8>;
  kernel<<<(unsigned)grid, 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? GDR_OK : GDR_CUDA_ERROR;
}

gdr_status ssm_step(const gdr_bf16* x, int64_t ldx, const void* dt, int dt_dtype, int64_t lddt, const float* A,
                    const gdr_bf16* B, int64_t ldb, const gdr_bf16* C, int64_t ldc, const float* D,
                    const float* dt_bias, int softplus, float* state, const int32_t* slots, int32_t NB, int32_t S,
                    int32_t H, int32_t P, int32_t G, int32_t NS, gdr_bf16* out, cudaStream_t stream) {
  if (dt_dtype != GDR_DTYPE_BF16 && dt_dtype != GDR_DTYPE_F32) return GDR_INVALID_ARG;
  SsmArgs a{};
  a.x = reinterpret_cast<const __nv_bfloat16*>(x);
  a.ldx = ldx;
  a.dt = dt;
  a.dt_f32 = dt_dtype == GDR_DTYPE_F32;
  a.lddt = lddt;
  a.A = A;
  a.B = reinterpret_cast<const __nv_bfloat16*>(B);
  a.C = reinterpret_cast<const __nv_bfloat16*>(C);
  a.ldb = ldb;
  a.ldc = ldc;
  a.D = D;
  a.dt_bias = dt_bias;
  a.softplus = softplus;
  a.H = H;
  a.P = P;
  a.G = G;
  a.NS = NS;
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.state = state;
  a.slots = slots;
  a.S = S;
  gdr_status rc = ssm_check(a, NB);
  if (rc != GDR_OK) return rc;
  if (S < 0 || (!slots && NB > S) || (S > 0 && !state)) return GDR_INVALID_ARG;
  if (NB == 0) return GDR_OK;
  if ((int64_t)NB * H > INT32_MAX) return GDR_INVALID_ARG;
  if ((rc = check_device()) != GDR_OK) return rc;
  ProfScope ps("ssm_step", stream, (double)NB * H);
  if (P % 4 == 0 && ((uintptr_t)state & 15) == 0) k_ssm_step<4><<<NB * H, 256, 0, stream>>>(a);
  else k_ssm_step<1><<<NB * H, 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? GDR_OK : GDR_CUDA_ERROR;
}

}  // extern "C"
