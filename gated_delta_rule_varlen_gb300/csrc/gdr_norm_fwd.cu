// gdr_norm_fwd.cu -- forward of the norms around a block (gdr_norm.cuh).
#include "gdr_norm.cuh"

namespace gdr {
namespace {

// Bound by HBM: each input read and each output written once.  Rows are dealt
// to the blocks in turn; rows past the end keep their threads in the barriers.
// Measured (BF16): 32768 x 48 rows of 128 with a gate 208 us (85% of the copy rate),
// 8191 rows of 2048 between two blocks 27 us (72%).  Rows ahead in shared memory took
// both directions together from 1015 to 550 us and from 130 to 93 us.
// Arithmetic in pairs of columns, so that its instructions fit beside the loads.
// OUT: the norm of a block's output alone (and its gate), without the residual
// and the second norm: fewer registers.
template <typename T, int V, int TPR, int NV, bool OUT, bool SHIFT>
struct FwdRows {
  static constexpr int ITEMS = (OUT ? 2 : 3) * NV, THREADS = norm_threads(TPR);
  static constexpr int DEPTH = rows_ahead(THREADS, ITEMS * V * (int)sizeof(T));
  static constexpr bool AHEAD = V * sizeof(T) >= 4 && DEPTH >= 1;  // (no copies of two bytes)
  using Rows = RowsAhead<T, AHEAD ? V : 8, ITEMS, DEPTH, THREADS, !SHIFT>;
};

template <typename T, int V, int TPR, int NV, bool CLUSTER, bool OUT, bool SHIFT>
__global__ void __launch_bounds__(norm_threads(TPR)) k_norm_fwd(NormArgs a) {
  using F = FwdRows<T, V, TPR, NV, OUT, SHIFT>;
  using Rows = typename F::Rows;
  constexpr bool AHEAD = F::AHEAD;
  constexpr int P = pairs_of<V>, DEPTH = F::DEPTH;
  __shared__ float2 sm[2][RowGroup<TPR, CLUSTER>::SUMS];
  const RowGroup<TPR, CLUSTER> g;
  // a shifted row's vectors start m elements before it, on 16 bytes
  const int m = SHIFT ? (int)(g.first % V) * (a.D % V) % V : 0;
  auto col = [&](int i) { return (i * g.lanes + g.lane) * V - m; };
  auto whole = [&](int i) { return !SHIFT || (col(i) >= 0 && col(i) + V <= a.D); };
  auto store = [&](T* row, int i, const uint64_t (&f)[P]) {
    if (whole(i)) store_pairs<T, V>(row + col(i), f);
    else store_clipped<T, V>(row, col(i), a.D, f);
  };
  const float inv_d = 1.f / (float)a.D;
  // The weights stay in registers, but for blocks that leave a thread 64 of them.
  constexpr bool KEEP = TPR < 1024;
  uint64_t wk[KEEP ? NV : 1][P], pk[KEEP ? NV : 1][P];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col(i);
      if (c < a.D) {
        if (!OUT && a.w) load_weight<T, V, SHIFT>(a, a.w, c, wk[i]);
        if (a.w_post) load_weight<T, V, SHIFT>(a, a.w_post, c, pk[i]);
      }
    }
  }
  auto weight = [&](const uint64_t (&kept)[KEEP ? NV : 1][P], const void* p, int i, uint64_t (&f)[P]) {
    if constexpr (KEEP) {
#pragma unroll
      for (int q = 0; q < P; ++q) f[q] = kept[i][q];
    } else {
      load_weight<T, V, SHIFT>(a, p, col(i), f);
    }
  };
  const bool has_res = !OUT && a.res.p, has_y = !OUT && a.y;
  extern __shared__ __align__(16) unsigned char norm_smem[];
  Rows ahead(norm_smem);
  Cursor<T, OUT ? 2 : 3> in(g.first, g.step, a.R1);  // the next row to ask for
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
          const int c = col(i);
          const int bytes = SHIFT ? min(V, a.D - c) * (int)sizeof(T) : V * (int)sizeof(T);
          if (c < a.D) {
            ahead.ask(slot, i, in.p[0] + c, bytes);
            if (a.gate.p) ahead.ask(slot, NV + i, in.p[1] + c, bytes);
            if constexpr (!OUT)
              if (has_res) ahead.ask(slot, 2 * NV + i, in.p[2] + c, bytes);
          }
        }
      }
      cp_async_commit();
    } else if (in.r < a.rows) {
      auto fetch = [&](bool given, int k, auto& to) {
        if (!given) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = col(i);
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
  for (int64_t r = g.first; r - g.grp < a.rows; r += g.step) {
    const bool live = r < a.rows;
    if constexpr (AHEAD) cp_async_wait<DEPTH - 1>();
    else ask(0);
    // vector i of a tensor: from shared memory whenever it is used, or registers
    auto get = [&](int k, int i, const Vec<T, V>& held, uint64_t (&f)[P]) {
      if constexpr (AHEAD) to_pairs<T, V>(ahead.get(slot, k * NV + i), f);
      else to_pairs<T, V>(held, f);
      if (SHIFT && !whole(i)) clip_pairs<V>(f, col(i), a.D);
    };
    auto put = [&](void* to, const uint64_t (&f)[NV][P]) {
      if (!to || !live) return;
      T* p = static_cast<T*>(to) + r * a.D;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < a.D) store(p, i, f[i]);
    };
    auto mean_square = [&](const uint64_t (&f)[NV][P], float2* buf) {
      uint64_t s = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < P; ++q) s = fma2(f[i][q], f[i][q], s);
      float ss[1] = {sum_of(s)};
      g.sum(ss, buf);
      return fmaf(ss[0], inv_d, a.eps);
    };
    uint64_t u[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (live && col(i) < a.D) get(0, i, raw.x[i], u[i]);
      else zero_pairs<V>(u[i]);
    }
    if (a.w_post) {
      const uint64_t r1 = both(rsqrtf(mean_square(u, sm[0])));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (col(i) < a.D) {
          uint64_t w[P];
          weight(pk, a.w_post, i, w);
#pragma unroll
          for (int q = 0; q < P; ++q) u[i][q] = mul2(u[i][q], mul2(r1, w[q]));
        }
      }
    }
    if (a.gate.p && live) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < a.D) {
          uint64_t z[P], sg, act;
          get(1, i, raw.z[i], z);
#pragma unroll
          for (int q = 0; q < P; ++q) {
            gate_of<T>(z[q], sg, act, a.sigmoid);
            u[i][q] = mul2(u[i][q], act);
          }
        }
    }
    if (has_res && live) {
      const uint64_t alpha = both(a.alpha);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < a.D) {
          uint64_t r[P];
          get(2, i, raw.r[OUT ? 0 : i], r);
#pragma unroll
          for (int q = 0; q < P; ++q) u[i][q] = fma2(alpha, u[i][q], r[q]);
        }
    }
    put(a.h, u);
    if (has_y) {
      const uint64_t r2 = both(rsqrtf(mean_square(u, sm[1])));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (col(i) < a.D) {
          uint64_t w[P];
          weight(wk, a.w, i, w);
#pragma unroll
          for (int q = 0; q < P; ++q) u[i][q] = mul2(u[i][q], mul2(r2, w[q]));
        }
      }
      put(a.y, u);
    }
    // a row that runs only one of the two sums would meet its own buffer again
    if (!(a.w_post && has_y)) g.sync();
    if constexpr (AHEAD) {  // (what was read from the slot has been used)
      ask(slot);
      slot = slot == DEPTH - 1 ? 0 : slot + 1;
    }
  }
}

template <typename T, int V, int TPR, int NV, bool CLUSTER, bool OUT, bool SHIFT>
cudaError_t launch_one(const NormArgs& a, const NormShape& s, int* parts, cudaStream_t st) {
  static Held held;
  using F = FwdRows<T, V, TPR, NV, OUT, SHIFT>;
  const size_t smem = F::AHEAD ? F::Rows::BYTES : 0;
  return norm_launch(k_norm_fwd<T, V, TPR, NV, CLUSTER, OUT, SHIFT>, a, s, smem, 32, held, parts, st);
}

template <typename T, int VT>
cudaError_t launch_t(const NormArgs& a, const NormShape& s, int* parts, cudaStream_t st) {
  constexpr int N = 8 / VT;  // vectors of 8 elements
  const bool out = !a.res.p && !a.w;  // the norm of a block's output alone
#define GDR_NORM_CASE(v, tpr, nv, cl, sh)                                                 \
  if (s.V == v && s.TPR == tpr && s.NV == nv && (s.cluster > 0) == cl && s.shift == sh)   \
    return out ? launch_one<T, v, tpr, nv, cl, true, sh>(a, s, parts, st)                 \
               : launch_one<T, v, tpr, nv, cl, false, sh>(a, s, parts, st);
#define GDR_NORM_CASES(tpr, nv, cl)     \
  GDR_NORM_CASE(VT, tpr, nv, cl, false) \
  GDR_NORM_CASE(VT, tpr, nv, cl, true)
  GDR_NORM_CASES(2, 1, false)
  GDR_NORM_CASES(4, 1, false)
  GDR_NORM_CASES(8, 1, false)
  GDR_NORM_CASES(8, 2, false)
  GDR_NORM_CASES(16, 2, false)
  GDR_NORM_CASES(32, 2, false)
  GDR_NORM_CASES(64, 2, false)
  GDR_NORM_CASES(96, 2, false)
  GDR_NORM_CASES(128, 2, false)
  if constexpr (VT == 4) {  // (of 16 bits 128 threads with two vectors hold as much)
    GDR_NORM_CASES(256, N, false)
  }
  GDR_NORM_CASES(384, N, false)
  GDR_NORM_CASES(512, N, false)
  GDR_NORM_CASES(640, N, false)
  GDR_NORM_CASES(768, N, false)
  GDR_NORM_CASES(1024, N, false)
  GDR_NORM_CASES(128, 2, true)
  GDR_NORM_CASE(1, 32, 8, false, false)
  GDR_NORM_CASE(1, 128, 8, true, false)
#undef GDR_NORM_CASES
#undef GDR_NORM_CASE
  return cudaErrorInvalidConfiguration;
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, int dtype, const NormShape& s, cudaStream_t st) {
  int parts = 0;
  switch (dtype) {
    case GDR_DTYPE_BF16: return launch_t<__nv_bfloat16, 8>(a, s, &parts, st);
    case GDR_DTYPE_F16: return launch_t<__half, 8>(a, s, &parts, st);
    default: return launch_t<float, 4>(a, s, &parts, st);
  }
}

}  // namespace gdr
