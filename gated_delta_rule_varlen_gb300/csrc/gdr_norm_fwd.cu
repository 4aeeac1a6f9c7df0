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
  RowIndex row((int64_t)blockIdx.x * G::GROUPS + grp, (int64_t)gridDim.x * G::GROUPS, a.R1);
  struct Raw {
    Vec<T, V> x[NV], z[NV], r[OUT ? 1 : NV];
  };
  auto ask = [&](const RowIndex& at, Raw& raw) {
    if (at.r >= a.rows) return;
    const T* xp = at.template of<T>(a.x);
    const T* zp = a.gate.p ? at.template of<T>(a.gate) : nullptr;
    const T* rp = has_res ? at.template of<T>(a.res) : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      if (c < a.D) {
        raw.x[i] = vload<T, V>(xp + c);
        if (zp) raw.z[i] = vload<T, V>(zp + c);
        if (rp) raw.r[OUT ? 0 : i] = vload<T, V>(rp + c);
      }
    }
  };
  // Rows are asked for ahead where two at least fit 40 KB a block: with the row in
  // work alone too few bytes are in flight.
  constexpr int ITEMS = (OUT ? 2 : 3) * NV, SLOT = ITEMS * G::THREADS * 16;
  constexpr int DEPTH = SLOT > 20480 ? 1 : SLOT * 4 <= 40960 ? 4 : 40960 / SLOT;
  constexpr bool AHEAD = V > 1 && DEPTH >= 2;
  using Ahead = RowsAhead<T, (V > 1 ? V : 4), ITEMS, DEPTH, G::THREADS>;
  __shared__ __align__(16) unsigned char ahead[AHEAD ? Ahead::BYTES : 16];
  Ahead rows(ahead);
  auto ask_ahead = [&](const RowIndex& at, int slot) {
    if constexpr (AHEAD) {
      if (at.r < a.rows) {
        const T* xp = at.template of<T>(a.x);
        const T* zp = a.gate.p ? at.template of<T>(a.gate) : nullptr;
        const T* rp = has_res ? at.template of<T>(a.res) : nullptr;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (i * TPR + lane) * V;
          if (c < a.D) {
            rows.ask(slot, i, xp + c);
            if (zp) rows.ask(slot, NV + i, zp + c);
            if constexpr (!OUT)
              if (rp) rows.ask(slot, 2 * NV + i, rp + c);
          }
        }
      }
      cp_async_commit();
    }
  };
  Raw raw;
  RowIndex far = row;
  if constexpr (AHEAD) {
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
      ask_ahead(far, i);
      far.next();
    }
  }
  int slot = 0;
#pragma unroll 1
  for (; row.r - grp < a.rows; row.next()) {
    const bool live = row.r < a.rows;
    if constexpr (AHEAD) cp_async_wait<DEPTH - 1>();
    else ask(row, raw);
    // the row's vectors: from shared memory whenever they are used, or registers
    auto vec = [&](int item, const Vec<T, V>& held) {
      if constexpr (AHEAD) return rows.get(slot, item);
      else return held;
    };
    auto put = [&](void* to, const uint64_t (&f)[NV][P]) {
      if (!to || !live) return;
      T* p = static_cast<T*>(to) + row.r * a.D;
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
      ask_ahead(far, slot);
      far.next();
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
