// gdr_norm_fwd.cu -- forward of the norms around a block (gdr_norm.cuh).
#include "gdr_norm.cuh"

namespace gdr {
namespace {

// Bound by HBM: each input read and each output written once.  Rows are dealt
// to the blocks in turn; rows past the end keep their threads in the barriers.
// Threads of few columns keep their weights in registers over all their rows.
// Arithmetic in pairs of columns, so that its instructions fit beside the loads.
// OUT: the norm of a block's output alone (and its gate), without the residual
// and the second norm: fewer registers.
template <typename T, int V, int TPR, int NV, bool OUT>
__global__ void __launch_bounds__(norm_threads(TPR)) k_norm_fwd(NormArgs a) {
  using G = RowGroup<TPR>;
  constexpr int P = pairs_of<V>;
  constexpr bool KEEP = NV * V <= 16;
  __shared__ float2 sm[2][G::WARPS];
  const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const float inv_d = 1.f / (float)a.D;
  uint64_t wk[KEEP ? NV : 1][P], pk[KEEP ? NV : 1][P];
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
  const bool has_res = !OUT && a.res.p, has_y = !OUT && a.y;
  // Rows are asked for ahead where two at least fit 40 KB a block: with the row in
  // work alone too few bytes are in flight.
  constexpr int ITEMS = (OUT ? 2 : 3) * NV, SLOT = ITEMS * G::THREADS * 16;
  constexpr int DEPTH = SLOT > 20480 ? 1 : SLOT * 4 <= 40960 ? 4 : 40960 / SLOT;
  constexpr bool AHEAD = V > 1 && DEPTH >= 2;
  using Ahead = RowsAhead<T, (V > 1 ? V : 4), ITEMS, DEPTH, G::THREADS>;
  __shared__ __align__(16) unsigned char ahead_rows[AHEAD ? Ahead::BYTES : 16];
  Ahead ahead(ahead_rows);
  const int64_t first = (int64_t)blockIdx.x * G::GROUPS + grp, step = (int64_t)gridDim.x * G::GROUPS;
  Cursor<T, OUT ? 2 : 3> in(first, step, a.R1);  // the next row to ask for
  in.add(0, a.x);
  in.add(1, a.gate);
  if constexpr (!OUT) in.add(2, a.res);
  struct Raw {
    Vec<T, V> x[NV], z[NV], r[OUT ? 1 : NV];
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
            if constexpr (!OUT)
              if (has_res) ahead.ask(slot, 2 * NV + i, in.p[2] + c);
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
      if constexpr (!OUT) fetch(has_res, 2, raw.r);
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
    auto mean_square = [&](const uint64_t (&f)[NV][P], float2* buf) {
      uint64_t s = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < P; ++q) s = fma2(f[i][q], f[i][q], s);
      float ss = sum_of(s);
      G::sum(ss, buf);
      return fmaf(ss, inv_d, a.eps);
    };
    uint64_t u[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (live && (i * TPR + lane) * V < a.D) to_pairs<T, V>(vec(i, raw.x[i]), u[i]);
      else zero_pairs<V>(u[i]);
    }
    if (a.w_post) {
      const uint64_t r1 = both(rsqrtf(mean_square(u, sm[0])));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * V;
        if (c < a.D) {
          uint64_t w[P];
          if constexpr (!KEEP) load_weight<T, V>(a, a.w_post, c, w);
#pragma unroll
          for (int q = 0; q < P; ++q) u[i][q] = mul2(u[i][q], mul2(r1, KEEP ? pk[KEEP ? i : 0][q] : w[q]));
        }
      }
    }
    if (a.gate.p && live) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((i * TPR + lane) * V < a.D) {
          uint64_t z[P], sg, act;
          to_pairs<T, V>(vec(NV + i, raw.z[i]), z);
#pragma unroll
          for (int q = 0; q < P; ++q) {
            gate_of(z[q], sg, act, a.sigmoid);
            u[i][q] = mul2(u[i][q], act);
          }
        }
    }
    if (has_res && live) {
      const uint64_t alpha = both(a.alpha);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((i * TPR + lane) * V < a.D) {
          uint64_t r[P];
          to_pairs<T, V>(vec(2 * NV + i, raw.r[OUT ? 0 : i]), r);
#pragma unroll
          for (int q = 0; q < P; ++q) u[i][q] = fma2(alpha, u[i][q], r[q]);
        }
    }
    put(a.h, u);
    if (has_y) {
      const uint64_t r2 = both(rsqrtf(mean_square(u, sm[1])));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * V;
        if (c < a.D) {
          uint64_t w[P];
          if constexpr (!KEEP) load_weight<T, V>(a, a.w, c, w);
#pragma unroll
          for (int q = 0; q < P; ++q) u[i][q] = mul2(u[i][q], mul2(r2, KEEP ? wk[KEEP ? i : 0][q] : w[q]));
        }
      }
      put(a.y, u);
    }
    // a row that runs only one of the two sums would meet its own buffer again
    if (TPR > 32 && !(a.w_post && has_y)) __syncthreads();
    if constexpr (AHEAD) {  // (what was read from the slot has been used)
      ask(slot);
      slot = slot == DEPTH - 1 ? 0 : slot + 1;
    }
  }
}

template <typename T, int VT>
cudaError_t launch_t(const NormArgs& a, const NormShape& s, cudaStream_t st) {
#define GDR_NORM_CASE(v, tpr, nv)                                                                              \
  if (s.V == v && s.TPR == tpr && s.NV == nv) {                                                                \
    constexpr int groups = RowGroup<tpr>::GROUPS, threads = norm_threads(tpr);                                 \
    const int64_t work = (a.rows + groups - 1) / groups;                                                       \
    static int occ = 0, occ_out = 0;                                                                           \
    if (a.res.p || a.w) {                                                                                      \
      const int blocks = norm_grid(k_norm_fwd<T, v, tpr, nv, false>, threads, 0, work, 32, &occ);              \
      k_norm_fwd<T, v, tpr, nv, false><<<blocks, threads, 0, st>>>(a);                                         \
    } else {                                                                                                   \
      const int blocks = norm_grid(k_norm_fwd<T, v, tpr, nv, true>, threads, 0, work, 32, &occ_out);           \
      k_norm_fwd<T, v, tpr, nv, true><<<blocks, threads, 0, st>>>(a);                                          \
    }                                                                                                          \
    return cudaGetLastError();                                                                                 \
  }
  GDR_NORM_CASE(VT, 8, 1)
  GDR_NORM_CASE(VT, 8, 2)
  GDR_NORM_CASE(VT, 16, 2)
  GDR_NORM_CASE(VT, 32, 2)
  GDR_NORM_CASE(VT, 32, 4)
  GDR_NORM_CASE(VT, 128, 2)
  GDR_NORM_CASE(VT, 256, 2)
  GDR_NORM_CASE(VT, 512, 2)
  GDR_NORM_CASE(VT, 512, 4)
  GDR_NORM_CASE(VT, 1024, 4)
  GDR_NORM_CASE(1, 32, 8)
  GDR_NORM_CASE(1, 256, 8)
  GDR_NORM_CASE(1, 1024, 16)
#undef GDR_NORM_CASE
  return cudaErrorInvalidConfiguration;
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, int dtype, const NormShape& s, cudaStream_t st) {
  switch (dtype) {
    case GDR_DTYPE_BF16: return launch_t<__nv_bfloat16, 8>(a, s, st);
    case GDR_DTYPE_F16: return launch_t<__half, 8>(a, s, st);
    default: return launch_t<float, 4>(a, s, st);
  }
}

}  // namespace gdr
