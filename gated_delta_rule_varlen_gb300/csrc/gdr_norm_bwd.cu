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

// Blocks an SM holds at least (which bounds the registers): rows of 8 elements a
// thread take about 90 of them, of 16 about 160.
constexpr int norm_bwd_min_blocks(int TPR, int elements, bool out) {
  if (TPR > 32) return TPR > 384 ? 1 : TPR > 128 ? 2 : TPR == 128 ? 3 : TPR == 96 ? 4 : 6;
  return elements <= 8 ? 5 : out ? 4 : 3;
}

// Bound by HBM.  A block keeps its columns' weight gradients in registers over
// all its rows and leaves one partial row; k_norm_wgrad adds those.  OUT: as in
// the forward.  Measured (BF16): 32768 x 48 rows of 128 with a gate 321 us (92% of the
// copy rate), 8191 rows of 2048 between two blocks 55 us (53%).
template <typename T, int V, int TPR, int NV, bool OUT, bool SHIFT>
struct BwdRows {
  static constexpr int ITEMS = (OUT ? 3 : 5) * NV, THREADS = norm_threads(TPR);
  static constexpr int DEPTH = rows_ahead(THREADS, ITEMS * V * (int)sizeof(T));
  static constexpr bool AHEAD = V * sizeof(T) >= 4 && DEPTH >= 1;  // (no copies of two bytes)
  using Rows = RowsAhead<T, AHEAD ? V : 8, ITEMS, DEPTH, THREADS, !SHIFT>;
};

template <typename T, int V, int TPR, int NV, bool CLUSTER, bool OUT, bool SHIFT>
__global__ void __launch_bounds__(norm_threads(TPR), norm_bwd_min_blocks(TPR, V * NV, OUT)) k_norm_bwd(NormArgs a) {
  using F = BwdRows<T, V, TPR, NV, OUT, SHIFT>;
  using Rows = typename F::Rows;
  constexpr bool AHEAD = F::AHEAD;
  constexpr int P = pairs_of<V>, DEPTH = F::DEPTH;
  __shared__ float2 sm[3][RowGroup<TPR, CLUSTER>::SUMS];
  next_may_start();  // (the sum of the partial rows)
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
  const uint64_t one = both(1.f), minus = both(-1.f);
  const bool has_res = !OUT && a.res.p, has_dy = !OUT && a.dy.p;
  uint64_t dw[OUT ? 1 : NV][P], dwp[NV][P];
  // The weights stay in registers, but for blocks that leave a thread 64 of them.
  constexpr bool KEEP = TPR < 1024;
  uint64_t wk[KEEP ? NV : 1][P], pk[KEEP ? NV : 1][P];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    zero_pairs<V>(dw[OUT ? 0 : i]);
    zero_pairs<V>(dwp[i]);
  }
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
  extern __shared__ __align__(16) unsigned char norm_smem[];
  Rows ahead(norm_smem);
  Cursor<T, OUT ? 3 : 5> in(g.first, g.step, a.R1);  // the next row to ask for
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
          const int c = col(i);
          const int bytes = SHIFT ? min(V, a.D - c) * (int)sizeof(T) : V * (int)sizeof(T);
          if (c < a.D) {
            ahead.ask(slot, i, in.p[0] + c, bytes);
            if (a.gate.p) ahead.ask(slot, NV + i, in.p[1] + c, bytes);
            if (a.dh.p) ahead.ask(slot, 2 * NV + i, in.p[2] + c, bytes);
            if constexpr (!OUT) {
              if (has_dy) ahead.ask(slot, 3 * NV + i, in.p[3] + c, bytes);
              if (has_dy && has_res) ahead.ask(slot, 4 * NV + i, in.p[4] + c, bytes);
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
          const int c = col(i);
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
    auto on = [&](int i) { return live && col(i) < a.D; };
    // r1
    float r1 = 1.f;
    if (a.w_post) {
      uint64_t s2 = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (on(i)) {
          uint64_t x[P];
          get(0, i, raw.x[i], x);
#pragma unroll
          for (int q = 0; q < P; ++q) s2 = fma2(x[q], x[q], s2);
        }
      float s[1] = {sum_of(s2)};
      g.sum(s, sm[0]);
      r1 = rsqrtf(fmaf(s[0], inv_d, a.eps));
    }
    const uint64_t rr1 = both(r1);
    // du starts as dH: dh and, through the second norm, dy
    uint64_t du[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (on(i) && a.dh.p) get(2, i, raw.h[i], du[i]);
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
          get(0, i, raw.x[i], h[i]);
          if (a.w_post) {
            weight(pk, a.w_post, i, f);
#pragma unroll
            for (int q = 0; q < P; ++q) h[i][q] = mul2(h[i][q], mul2(rr1, f[q]));
          }
          if (a.gate.p) {
            uint64_t sg, act;
            get(1, i, raw.z[i], f);
#pragma unroll
            for (int q = 0; q < P; ++q) {
              gate_of<T>(f[q], sg, act, a.sigmoid);
              h[i][q] = mul2(h[i][q], act);
            }
          }
          if (has_res) {
            get(4, i, raw.r[OUT ? 0 : i], f);
#pragma unroll
            for (int q = 0; q < P; ++q) h[i][q] = fma2(alpha, h[i][q], f[q]);
          }
          weight(wk, a.w, i, f);
          get(3, i, raw.y[OUT ? 0 : i], y);
#pragma unroll
          for (int q = 0; q < P; ++q) {
            s2 = fma2(h[i][q], h[i][q], s2);
            t2 = fma2(mul2(y[q], f[q]), h[i][q], t2);
          }
        }
      }
      float s[2] = {sum_of(s2), sum_of(t2)};
      g.sum(s, sm[1]);
      const float r2 = rsqrtf(fmaf(s[0], inv_d, a.eps));
      const float c2 = s[1] * r2 * inv_d;  // mean(dn hn)
      // du += r2 (dn - hn c2); a single column: r2 dn eps r2^2
      const uint64_t pa = both(a.D > 1 ? r2 : r2 * a.eps * r2 * r2), pb = both(a.D > 1 ? -r2 * r2 * c2 : 0.f);
      const uint64_t rr2 = both(r2);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (on(i)) {
          uint64_t f[P], y[P];
          weight(wk, a.w, i, f);
          get(3, i, raw.y[OUT ? 0 : i], y);
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
          get(1, i, raw.z[i], z);
          get(0, i, raw.x[i], n);
          if (a.w_post) {
            weight(pk, a.w_post, i, p);
#pragma unroll
            for (int q = 0; q < P; ++q) n[q] = mul2(n[q], mul2(rr1, p[q]));
          }
#pragma unroll
          for (int q = 0; q < P; ++q) {
            gate_of<T>(z[q], sg, act, a.sigmoid);
            // silu: sg + act (1 - sg); sigmoid: sg (1 - sg)
            const uint64_t rest = fma2(minus, sg, one);
            const uint64_t dact = a.sigmoid ? mul2(sg, rest) : fma2(act, rest, sg);
            n[q] = mul2(mul2(du[i][q], n[q]), dact);
            du[i][q] = mul2(du[i][q], act);
          }
          if (a.dgate) store(static_cast<T*>(a.dgate) + r * a.D, i, n);
        }
    }
    if (a.w_post) {
      uint64_t s2 = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (on(i)) {
          uint64_t x[P], p[P];
          get(0, i, raw.x[i], x);
          weight(pk, a.w_post, i, p);
#pragma unroll
          for (int q = 0; q < P; ++q) {
            x[q] = mul2(x[q], rr1);
            dwp[i][q] = fma2(du[i][q], x[q], dwp[i][q]);
            du[i][q] = mul2(du[i][q], p[q]);
            s2 = fma2(du[i][q], x[q], s2);
          }
        }
      float s[1] = {sum_of(s2)};
      g.sum(s, sm[2]);
      const float c1 = s[0] * inv_d;  // mean(dm xn)
      // dx = r1 (dm - xn c1); a single column: r1 dm eps r1^2
      const uint64_t pa = both(a.D > 1 ? r1 : r1 * a.eps * r1 * r1), pb = both(a.D > 1 ? -r1 * r1 * c1 : 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (on(i)) {
          uint64_t x[P];
          get(0, i, raw.x[i], x);
#pragma unroll
          for (int q = 0; q < P; ++q) du[i][q] = fma2(pa, du[i][q], mul2(pb, x[q]));
        }
    }
    put(a.dx, du);
    // rows that run one sum only would meet its buffer again
    if (!a.w_post) g.sync();
    if constexpr (AHEAD) {  // (what was read from the slot has been used)
      ask(slot);
      slot = slot == DEPTH - 1 ? 0 : slot + 1;
    }
  }
  if constexpr (AHEAD) cp_async_wait<0>();
  float* part = a.part + (int64_t)(blockIdx.x / g.cluster) * 2 * a.D;
  auto leave = [&](const uint64_t (&sums)[NV][P], float* to) {
    float* at = to;
    if constexpr (g.GROUPS > 1) {  // the groups' rows meet in shared memory, [GROUPS][D]
      __syncthreads();
      at = reinterpret_cast<float*>(norm_smem) + g.grp * a.D;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col(i);
      float f[V + 1];
#pragma unroll
      for (int q = 0; q < P; ++q) unpack2(sums[i][q], f[2 * q], f[2 * q + 1]);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (SHIFT ? c + v >= 0 && c + v < a.D : c < a.D) at[c + v] = f[v];
    }
    if constexpr (g.GROUPS > 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < a.D; c += g.THREADS) {
        float sum = 0.f;
        for (int j = 0; j < g.GROUPS; ++j) sum += reinterpret_cast<const float*>(norm_smem)[j * a.D + c];
        to[c] = sum;
      }
    }
  };
  if constexpr (!OUT)
    if (a.w) leave(dw, part);
  if (a.w_post) leave(dwp, part + a.D);
}

// dw and dw_post: the row groups' partial rows added in a fixed order.
__global__ void __launch_bounds__(1024) k_norm_wgrad(const float* __restrict__ part, int blocks, int D, float* dw,
                                                     float* dwp) {
  float* to = blockIdx.y == 0 ? dw : dwp;
  previous_ended();
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

template <typename T, int V, int TPR, int NV, bool CLUSTER, bool OUT, bool SHIFT>
cudaError_t launch_one(const NormArgs& a, const NormShape& s, int* parts, cudaStream_t st) {
  static Held held;
  using F = BwdRows<T, V, TPR, NV, OUT, SHIFT>;
  // (the groups' weight gradients meet in the same bytes: at most V NV columns a thread)
  const size_t smem = std::max((size_t)(F::AHEAD ? F::Rows::BYTES : 0), TPR <= 32 ? 128 * V * NV * sizeof(float) : (size_t)0);
  return norm_launch(k_norm_bwd<T, V, TPR, NV, CLUSTER, OUT, SHIFT>, a, s, smem, norm_bwd_blocks(a.D), held, parts, st);
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

cudaError_t launch_norm_bwd(const NormArgs& a, int dtype, const NormShape& s, int* parts, cudaStream_t st) {
  switch (dtype) {
    case GDR_DTYPE_BF16: return launch_t<__nv_bfloat16, 8>(a, s, parts, st);
    case GDR_DTYPE_F16: return launch_t<__half, 8>(a, s, parts, st);
    default: return launch_t<float, 4>(a, s, parts, st);
  }
}

namespace {

// Most row groups of a backward: the partial rows its workspace has to hold.
int max_norm_parts(int D) { return 152 * norm_bwd_blocks(D); }

// Rows of D elements: how they can be read.
struct RowLayout {
  int64_t R0;
  int R1, D, V;
  bool pieces = true, dense = true;  // in pieces of V = 16 bytes; one after another from 16 bytes on
  void input(const RowTensor& t) {
    if (!t.p) return;
    const bool on16 = ((uintptr_t)t.p & 15) == 0;
    pieces = pieces && on16 && t.s0 % V == 0 && t.s1 % V == 0;
    dense = dense && on16 && (R1 == 1 || t.s1 == D) && (R0 == 1 || t.s0 == (int64_t)R1 * D);
  }
  void output(const void* p) {
    pieces = pieces && ((uintptr_t)p & 15) == 0;
    dense = dense && ((uintptr_t)p & 15) == 0;
  }
};

// The threads that hold a row: in pieces of 16 bytes where all rows start on them,
// or, rows of any length that lie one after another, shifted to the 16 bytes each
// starts in; else (strided rows of odd places) single elements.  Fractions of the
// copy rate, forward / backward of the norms between two blocks in BF16, 2^27
// elements: shifted 0.32 / 0.21 at 66 columns and 0.49 / 0.32 at 1021, one by one
// 0.15 / 0.06 and 0.23 / 0.11.  Two pieces a thread up to 128 threads (what a row costs
// beside its elements is shared by 16 of BF16): 0.79 / 0.70 at 2048 columns.  Wider rows
// have 8 elements a thread, whose registers (90 in the backward) let an SM hold 768
// threads: 0.57 / 0.49 at 4096, with two pieces 0.54 / 0.31, as a cluster of two blocks
// 0.64 / 0.39, of FP32 0.86 / 0.83 against 0.66 / 0.56.  Past 1024 threads clusters: 0.48 /
// 0.31 at 16384, one block of four pieces a thread 0.51 / 0.18.
NormShape norm_shape(const RowLayout& l) {
  const int V = l.V, D = l.D, N = 8 / V;
  const bool shift = !(l.pieces && D % V == 0);
  if (!shift || l.dense) {
    const int n = shift ? (D + 2 * V - 2) / V : D / V;
    if (n <= 2) return {V, 2, 1, 0, shift};
    if (n <= 4) return {V, 4, 1, 0, shift};
    for (int tpr = 8; tpr <= 1024; tpr += tpr < 64 ? tpr : tpr < 128 ? 32 : tpr < 768 ? 128 : 256) {
      if (tpr == 8 && n <= 8) return {V, 8, 1, 0, shift};
      const int nv = tpr <= 128 ? 2 : N;
      if (n <= tpr * nv) return {V, tpr, nv, 0, shift};
    }
    const int cluster = (n + 255) / 256;
    if (cluster <= MAX_CLUSTER) return {V, 128, 2, cluster, shift};
  }
  if (D <= 256) return {1, 32, 8, 0, false};
  return {1, 128, 8, (D + 1023) / 1024, false};
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
  *scratch_bytes = (size_t)max_norm_parts(D) * 2 * D * sizeof(float);
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
  RowLayout l{R0, R1, D, dtype == GDR_DTYPE_F32 ? 4 : 8};
  for (const RowTensor& t : {a.x, a.gate, a.res}) l.input(t);
  for (const void* p : {h, y}) l.output(p);
  const NormShape s = norm_shape(l);
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
  RowLayout l{R0, R1, D, dtype == GDR_DTYPE_F32 ? 4 : 8};
  for (const RowTensor& t : {a.x, a.gate, a.res, a.dh, a.dy}) l.input(t);
  for (const void* p : {dx, dgate, dresidual}) l.output(p);
  const NormShape s = norm_shape(l);
  int parts = 0;
  if (a.rows > 0) {
    ProfScope ps("norm_bwd", stream, (double)a.rows * D);
    if (launch_norm_bwd(a, dtype, s, &parts, stream) != cudaSuccess) return GDR_CUDA_ERROR;
  }
  if (dweight || dpost_weight) {
    ProfScope ps("norm_wgrad", stream);
    if (launch_early(k_norm_wgrad, dim3((D + 31) / 32, 2), 1024, 0, stream, a.part, parts, D, dweight, dpost_weight) != cudaSuccess)
      return GDR_CUDA_ERROR;
  }
  return GDR_OK;
}

}  // extern "C"
