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
// all its rows and leaves one partial row; k_norm_wgrad adds those.  Threads of
// few columns keep the weights in registers too.  OUT: as in the forward.
template <typename T, int V, int TPR, int NV, bool OUT>
__global__ void __launch_bounds__(norm_threads(TPR), NV * V <= 8 ? (TPR <= 128 ? 5 : TPR == 256 ? 2 : 1) : NV * V == 16 ? (TPR <= 32 && OUT ? 4 : TPR <= 128 ? 3 : 1) : 1)
    k_norm_bwd(NormArgs a) {
  using G = RowGroup<TPR>;
  constexpr int P = pairs_of<V>;
  constexpr bool KEEP = NV * V <= 16;
  __shared__ float2 sm[3][G::WARPS];
  extern __shared__ float sred[];  // [GROUPS][D] when a block works on several rows
  const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const float inv_d = 1.f / (float)a.D;
  const uint64_t one = both(1.f), minus = both(-1.f);
  const bool has_res = !OUT && a.res.p, has_dy = !OUT && a.dy.p;
  uint64_t dw[OUT ? 1 : NV][P], dwp[NV][P];
  uint64_t wk[KEEP ? NV : 1][P], pk[KEEP ? NV : 1][P];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    zero_pairs<V>(dw[OUT ? 0 : i]);
    zero_pairs<V>(dwp[i]);
  }
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      if (c < a.D) {
        if (!OUT && a.w) load_weight<T, V>(a, a.w, c, wk[i]);
        if (a.w_post) load_weight<T, V>(a, a.w_post, c, pk[i]);
      }
    }
  }
  // weight vector i of this thread
  auto weight = [&](const uint64_t (&kept)[KEEP ? NV : 1][P], const void* p, int i, uint64_t (&f)[P]) {
    if constexpr (KEEP) {
#pragma unroll
      for (int q = 0; q < P; ++q) f[q] = kept[i][q];
    } else {
      load_weight<T, V>(a, p, (i * TPR + lane) * V, f);
    }
  };
  // Rows are asked for ahead where two at least fit 40 KB a block: with the row in
  // work alone too few bytes are in flight.
  constexpr int ITEMS = (OUT ? 3 : 5) * NV, SLOT = ITEMS * G::THREADS * 16;
  constexpr int DEPTH = SLOT > 20480 ? 1 : SLOT * 4 <= 40960 ? 4 : 40960 / SLOT;
  constexpr bool AHEAD = V > 1 && DEPTH >= 2;
  using Ahead = RowsAhead<T, (V > 1 ? V : 4), ITEMS, DEPTH, G::THREADS>;
  __shared__ __align__(16) unsigned char ahead_rows[AHEAD ? Ahead::BYTES : 16];
  Ahead ahead(ahead_rows);
  const int64_t first = (int64_t)blockIdx.x * G::GROUPS + grp, step = (int64_t)gridDim.x * G::GROUPS;
  Cursor<T, OUT ? 3 : 5> in(first, step, a.R1);  // the next row to ask for
  in.add(0, a.x);
  in.add(1, a.gate);
  in.add(2, a.dh);
  if constexpr (!OUT) {
    in.add(3, a.dy);
    in.add(4, a.res);
  }
  struct Raw {
    Vec<T, V> x[NV], z[NV], h[NV], r[OUT ? 1 : NV], y[OUT ? 1 : NV];
  };
  Raw raw;
  auto ask = [&](int slot) {
    if constexpr (AHEAD) {
      if (in.r < a.rows) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (i * TPR + lane) * V;
          if (c < a.D) {
            ahead.ask(slot, i, in.p[0] + c);
            if (a.gate.p) ahead.ask(slot, NV + i, in.p[1] + c);
            if (a.dh.p) ahead.ask(slot, 2 * NV + i, in.p[2] + c);
            if constexpr (!OUT) {
              if (has_dy) ahead.ask(slot, 3 * NV + i, in.p[3] + c);
              if (has_dy && has_res) ahead.ask(slot, 4 * NV + i, in.p[4] + c);
            }
          }
        }
      }
      cp_async_commit();
    } else if (in.r < a.rows) {
      auto fetch = [&](bool given, int k, auto& to) {
        if (!given) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (i * TPR + lane) * V;
          if (c < a.D) to[i] = vload<T, V>(in.p[k] + c);
        }
      };
      fetch(true, 0, raw.x);
      fetch(a.gate.p, 1, raw.z);
      fetch(a.dh.p, 2, raw.h);
      if constexpr (!OUT) {
        fetch(has_dy, 3, raw.y);
        fetch(has_dy && has_res, 4, raw.r);
      }
    }
    in.next();
  };
  if constexpr (AHEAD) {
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) ask(i);
  }
  int slot = 0;
#pragma unroll 1
  for (int64_t r = first; r - grp < a.rows; r += step) {
    const bool live = r < a.rows;
    if constexpr (AHEAD) cp_async_wait<DEPTH - 1>();
    else ask(0);
    // the row's vectors: from shared memory whenever they are used, or registers
    auto vec = [&](int item, const Vec<T, V>& held) {
      if constexpr (AHEAD) return ahead.get(slot, item);
      else return held;
    };
    auto put = [&](void* to, const uint64_t (&f)[NV][P]) {
      if (!to || !live) return;
      T* p = static_cast<T*>(to) + r * a.D;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * V;
        if (c < a.D) store_pairs<T, V>(p + c, f[i]);
      }
    };
    auto on = [&](int i) { return live && (i * TPR + lane) * V < a.D; };
    // r1
    float r1 = 1.f;
    if (a.w_post) {
      uint64_t s2 = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (on(i)) {
          uint64_t x[P];
          to_pairs<T, V>(vec(i, raw.x[i]), x);
#pragma unroll
          for (int q = 0; q < P; ++q) s2 = fma2(x[q], x[q], s2);
        }
      float s = sum_of(s2);
      G::sum(s, sm[0]);
      r1 = rsqrtf(fmaf(s, inv_d, a.eps));
    }
    const uint64_t rr1 = both(r1);
    // du starts as dH: dh and, through the second norm, dy
    uint64_t du[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (on(i) && a.dh.p) to_pairs<T, V>(vec(2 * NV + i, raw.h[i]), du[i]);
      else zero_pairs<V>(du[i]);
    }
    if (has_dy) {
      uint64_t h[NV][P], s2 = 0, t2 = 0;
      const uint64_t alpha = both(a.alpha);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        zero_pairs<V>(h[i]);
        if (on(i)) {
          uint64_t f[P], y[P];
          to_pairs<T, V>(vec(i, raw.x[i]), h[i]);
          if (a.w_post) {
            weight(pk, a.w_post, i, f);
#pragma unroll
            for (int q = 0; q < P; ++q) h[i][q] = mul2(h[i][q], mul2(rr1, f[q]));
          }
          if (a.gate.p) {
            uint64_t sg, act;
            to_pairs<T, V>(vec(NV + i, raw.z[i]), f);
#pragma unroll
            for (int q = 0; q < P; ++q) {
              gate_of(f[q], sg, act, a.sigmoid);
              h[i][q] = mul2(h[i][q], act);
            }
          }
          if (has_res) {
            to_pairs<T, V>(vec(4 * NV + i, raw.r[OUT ? 0 : i]), f);
#pragma unroll
            for (int q = 0; q < P; ++q) h[i][q] = fma2(alpha, h[i][q], f[q]);
          }
          weight(wk, a.w, i, f);
          to_pairs<T, V>(vec(3 * NV + i, raw.y[OUT ? 0 : i]), y);
#pragma unroll
          for (int q = 0; q < P; ++q) {
            s2 = fma2(h[i][q], h[i][q], s2);
            t2 = fma2(mul2(y[q], f[q]), h[i][q], t2);
          }
        }
      }
      float s = sum_of(s2), t = sum_of(t2);
      G::sum2(s, t, sm[1]);
      const float r2 = rsqrtf(fmaf(s, inv_d, a.eps));
      const float c2 = t * r2 * inv_d;  // mean(dn hn)
      // du += r2 (dn - hn c2); a single column: r2 dn eps r2^2
      const uint64_t pa = both(a.D > 1 ? r2 : r2 * a.eps * r2 * r2), pb = both(a.D > 1 ? -r2 * r2 * c2 : 0.f);
      const uint64_t rr2 = both(r2);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (on(i)) {
          uint64_t f[P], y[P];
          weight(wk, a.w, i, f);
          to_pairs<T, V>(vec(3 * NV + i, raw.y[OUT ? 0 : i]), y);
#pragma unroll
          for (int q = 0; q < P; ++q) {
            dw[OUT ? 0 : i][q] = fma2(y[q], mul2(h[i][q], rr2), dw[OUT ? 0 : i][q]);
            du[i][q] = fma2(pa, mul2(y[q], f[q]), fma2(pb, h[i][q], du[i][q]));
          }
        }
    }
    if (!OUT) put(a.dres, du);
    if (has_res) {
      const uint64_t alpha = both(a.alpha);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < P; ++q) du[i][q] = mul2(alpha, du[i][q]);
    }
    if (a.gate.p) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (on(i)) {
          uint64_t z[P], n[P], p[P], sg, act;
          to_pairs<T, V>(vec(NV + i, raw.z[i]), z);
          to_pairs<T, V>(vec(i, raw.x[i]), n);
          if (a.w_post) {
            weight(pk, a.w_post, i, p);
#pragma unroll
            for (int q = 0; q < P; ++q) n[q] = mul2(n[q], mul2(rr1, p[q]));
          }
#pragma unroll
          for (int q = 0; q < P; ++q) {
            gate_of(z[q], sg, act, a.sigmoid);
            // silu: sg + act (1 - sg); sigmoid: sg (1 - sg)
            const uint64_t rest = fma2(minus, sg, one);
            const uint64_t dact = a.sigmoid ? mul2(sg, rest) : fma2(act, rest, sg);
            n[q] = mul2(mul2(du[i][q], n[q]), dact);
            du[i][q] = mul2(du[i][q], act);
          }
          if (a.dgate) store_pairs<T, V>(static_cast<T*>(a.dgate) + r * a.D + (i * TPR + lane) * V, n);
        }
    }
    if (a.w_post) {
      uint64_t s2 = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (on(i)) {
          uint64_t x[P], p[P];
          to_pairs<T, V>(vec(i, raw.x[i]), x);
          weight(pk, a.w_post, i, p);
#pragma unroll
          for (int q = 0; q < P; ++q) {
            x[q] = mul2(x[q], rr1);
            dwp[i][q] = fma2(du[i][q], x[q], dwp[i][q]);
            du[i][q] = mul2(du[i][q], p[q]);
            s2 = fma2(du[i][q], x[q], s2);
          }
        }
      float s = sum_of(s2);
      G::sum(s, sm[2]);
      const float c1 = s * inv_d;  // mean(dm xn)
      // dx = r1 (dm - xn c1); a single column: r1 dm eps r1^2
      const uint64_t pa = both(a.D > 1 ? r1 : r1 * a.eps * r1 * r1), pb = both(a.D > 1 ? -r1 * r1 * c1 : 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (on(i)) {
          uint64_t x[P];
          to_pairs<T, V>(vec(i, raw.x[i]), x);
#pragma unroll
          for (int q = 0; q < P; ++q) du[i][q] = fma2(pa, du[i][q], mul2(pb, x[q]));
        }
    }
    put(a.dx, du);
    // rows that run one sum only would meet its buffer again
    if (TPR > 32 && !a.w_post) __syncthreads();
    if constexpr (AHEAD) {  // (what was read from the slot has been used)
      ask(slot);
      slot = slot == DEPTH - 1 ? 0 : slot + 1;
    }
  }
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.D;
  auto leave = [&](const uint64_t (&gp)[NV][P], float* to) {
    float g[NV][V + 1];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < P; ++q) unpack2(gp[i][q], g[i][2 * q], g[i][2 * q + 1]);
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
  if constexpr (!OUT)
    if (a.w) leave(dw, part);
  if (a.w_post) leave(dwp, part + a.D);
}

// dw and dw_post: the blocks' partial rows added in a fixed order.
__global__ void __launch_bounds__(1024) k_norm_wgrad(const float* __restrict__ part, int blocks, int D, float* dw,
                                                     float* dwp) {
  float* to = blockIdx.y == 0 ? dw : dwp;
  if (!to) return;
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (c < D) {
#pragma unroll 8
    for (int i = row; i < blocks; i += 32) sum += part[((int64_t)i * 2 + blockIdx.y) * D + c];
  }
  s[row][lane] = sum;
  __syncthreads();
  if (row == 0 && c < D) {
#pragma unroll
    for (int i = 1; i < 32; ++i) sum += s[i][lane];
    to[c] = sum;
  }
}

template <typename T, int VT>
cudaError_t launch_t(const NormArgs& a, const NormShape& s, int* blocks, cudaStream_t st) {
#define GDR_NORM_CASE(v, tpr, nv)                                                                              \
  if (s.V == v && s.TPR == tpr && s.NV == nv) {                                                                \
    constexpr int groups = RowGroup<tpr>::GROUPS, threads = norm_threads(tpr);                                 \
    const size_t sm = groups > 1 ? (size_t)groups * a.D * sizeof(float) : 0;                                   \
    const int64_t work = (a.rows + groups - 1) / groups;                                                       \
    constexpr int most = norm_blocks_per_sm(threads);                                                          \
    static int occ = 0, occ_out = 0;                                                                           \
    if (a.res.p || a.w) {                                                                                      \
      *blocks = norm_grid(k_norm_bwd<T, v, tpr, nv, false>, threads, sm, work, most, &occ);                    \
      k_norm_bwd<T, v, tpr, nv, false><<<*blocks, threads, sm, st>>>(a);                                       \
    } else {                                                                                                   \
      *blocks = norm_grid(k_norm_bwd<T, v, tpr, nv, true>, threads, sm, work, most, &occ_out);                 \
      k_norm_bwd<T, v, tpr, nv, true><<<*blocks, threads, sm, st>>>(a);                                        \
    }                                                                                                          \
    return cudaGetLastError();                                                                                 \
  }
  GDR_NORM_CASE(VT, 8, 1)
  GDR_NORM_CASE(VT, 8, 2)
  GDR_NORM_CASE(VT, 16, 2)
  GDR_NORM_CASE(VT, 32, 2)
  GDR_NORM_CASE(VT, 128, 1)
  GDR_NORM_CASE(VT, 128, 2)
  GDR_NORM_CASE(VT, 256, 2)
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

cudaError_t launch_norm_bwd(const NormArgs& a, int dtype, const NormShape& s, int* blocks, cudaStream_t st) {
  switch (dtype) {
    case GDR_DTYPE_BF16: return launch_t<__nv_bfloat16, 8>(a, s, blocks, st);
    case GDR_DTYPE_F16: return launch_t<__half, 8>(a, s, blocks, st);
    default: return launch_t<float, 4>(a, s, blocks, st);
  }
}

namespace {

// Most blocks of a backward on rows of D elements, over the shapes that such
// rows take: the partial rows its workspace has to hold.
int max_norm_blocks(int D) { return 152 * norm_blocks_per_sm(D <= 2048 ? 128 : 256); }

// Whether rows of D elements at these addresses and strides can be read in
// 16-byte pieces.
bool rows16(const RowTensor& t, int V) {
  return !t.p || (((uintptr_t)t.p & 15) == 0 && t.s0 % V == 0 && t.s1 % V == 0);
}

// The threads that hold a row: 16-byte pieces where all rows allow them, else
// single elements.  Two pieces a thread (what a row costs beside its elements is
// then shared by 16 of BF16) while the row's group has 128 threads at least, or
// less than a warp's; within a warp there is no barrier a row.
NormShape norm_shape(int D, int dtype, bool vec, bool bwd) {
  const int V = dtype == GDR_DTYPE_F32 ? 4 : 8;
  if (vec && D % V == 0) {
    const int n = D / V;
    if (n <= 8) return {V, 8, 1};
    if (n <= 16) return {V, 8, 2};
    if (n <= 32) return {V, 16, 2};
    if (n <= 64) return {V, 32, 2};
    if (n <= 128) return bwd ? NormShape{V, 128, 1} : NormShape{V, 32, 4};
    if (n <= 256) return {V, 128, 2};
    if (n <= 512) return {V, 256, 2};
    if (n <= 1024) return {V, 512, 2};
    if (n <= 2048) return bwd ? NormShape{V, 1024, 2} : NormShape{V, 512, 4};
    return {V, 1024, 4};
  }
  if (D <= 256) return {1, 32, 8};
  if (D <= 2048) return {1, 256, 8};
  return {1, 1024, 16};
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
  a.wvec = (((uintptr_t)post_weight | (uintptr_t)weight) & 15) == 0;
  a.sigmoid = act == GDR_ACT_SIGMOID;
  a.alpha = residual ? res_scale : 1.f;
  a.eps = eps;
  a.h = h;
  a.y = y;
  const int V = dtype == GDR_DTYPE_F32 ? 4 : 8;
  const bool vec = rows16(a.x, V) && rows16(a.gate, V) && rows16(a.res, V) &&
                   (((uintptr_t)h | (uintptr_t)y) & 15) == 0;
  const NormShape s = norm_shape(D, dtype, vec, false);
  ProfScope ps("norm_fwd", stream, (double)a.rows * D);
  return launch_norm_fwd(a, dtype, s, stream) == cudaSuccess ? GDR_OK : GDR_CUDA_ERROR;
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
  a.wvec = (((uintptr_t)post_weight | (uintptr_t)weight) & 15) == 0;
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
  const NormShape s = norm_shape(D, dtype, vec, true);
  int blocks = 0;
  if (a.rows > 0) {
    ProfScope ps("norm_bwd", stream, (double)a.rows * D);
    if (launch_norm_bwd(a, dtype, s, &blocks, stream) != cudaSuccess) return GDR_CUDA_ERROR;
  }
  if (dweight || dpost_weight) {
    ProfScope ps("norm_wgrad", stream);
    k_norm_wgrad<<<dim3((D + 31) / 32, 2), 1024, 0, stream>>>(a.part, blocks, D, dweight, dpost_weight);
    if (cudaGetLastError() != cudaSuccess) return GDR_CUDA_ERROR;
  }
  return GDR_OK;
}

}  // extern "C"
