// gdr_sconv.cu -- the short causal depthwise convolution in front of the
// recurrences, over packed documents:
//   z[t][c] = bias[c] + sum_{j<W} w[c][j] xx[t - (W-1) + j][c],  out = z or silu(z)
// where xx is x inside the document and, before its first token, the W - 1
// rows of the document's start state (or zero).  Backward:
//   dz = dout act'(z),  dxx[t] = sum_j w[c][j] dz[t + (W-1) - j]  (same document),
//   dw[c][j] = sum_t dz[t] xx[t - (W-1) + j],  dbias = sum_t dz[t].
#include "gdr_ops.cuh"
#include "gdr_runtime.h"

namespace gdr {
namespace {

struct ConvArgs {
  const void *x, *weight, *bias;
  int wf32;             // weight and bias in FP32 (else in the type of x)
  int64_t ldx;          // row stride of x (elements)
  const int* cu;
  int N, T, C;
  int silu;
  const void* s0;       // [N][W-1][C] or null
  void *out, *st;       // [T][C]; [N][W-1][C] or null
  int tile;             // tokens per tile
  int cblocks;          // blocks along the channels; block b works on tile b / cblocks
};

// The filters of V channels from c on, one pair vector a tap, and their biases.
template <typename T, int V, int W>
__device__ __forceinline__ void load_filters(const ConvArgs& a, int c, uint64_t (&w)[W][pairs_of<V>],
                                             uint64_t (&b)[pairs_of<V>]) {
  auto at = [&](const void* p, int64_t i) { return load_param<T>(p, a.wf32, i); };
#pragma unroll
  for (int i = 0; i < pairs_of<V>; ++i) {
    const bool two = 2 * i + 1 < V;
    b[i] = a.bias ? pack2(at(a.bias, c + 2 * i), two ? at(a.bias, c + 2 * i + 1) : 0.f) : 0;
#pragma unroll
    for (int j = 0; j < W; ++j)
      w[j][i] = pack2(at(a.weight, (int64_t)(c + 2 * i) * W + j),
                      two ? at(a.weight, (int64_t)(c + 2 * i + 1) * W + j) : 0.f);
  }
}
// The W - 1 rows before token t of document d, which starts at ds.
template <typename T, int V, int W>
__device__ __forceinline__ void load_window(const ConvArgs& a, const T* x, const T* s0, int d, int ds, int t,
                                            uint64_t (&win)[W - 1][pairs_of<V>]) {
  constexpr int K = W - 1;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int p = t - K + k;
    if (p >= ds) to_pairs<T, V>(vload<T, V>(x + (int64_t)p * a.ldx), win[k]);
    else if (s0) to_pairs<T, V>(vload<T, V>(s0 + ((int64_t)d * K + (p - ds + K)) * a.C), win[k]);
    else zero_pairs<V>(win[k]);
  }
}

// Rows of the walks asked for ahead: in shared memory (4 to 16 bytes each a thread),
// or, single elements of 16 bits, which cannot be copied there, in registers.  (Of
// single FP32 elements the forward keeps its rows in registers, too: 65536 x 4095
// took 391 us against 465; the backward, with two rings, 785 against 918.  With the
// sigmoid of FP32 exact to 6e-7 the kept ones take 408 and 816.)
constexpr int kDepth = 8;
template <typename T, int V>
constexpr bool kRing = V * sizeof(T) >= 4;

// One thread owns V adjacent channels and walks the tokens of one tile with
// the last W - 1 inputs in registers, so each input is read once (and W - 1
// rows again at a tile's start).  Arithmetic in pairs of channels: the kernel is
// bound by HBM (2 accesses an element) only while its instructions fit beside.
// Measured (BF16, 4 taps, silu): 32768 tokens x 10240 channels 214 us = 92% of the copy
// rate (one row at a time, without rows ahead, 261); 65536 tokens in pieces of 16 bytes
// (8192 channels) 331 us, in pairs of channels (8190) 489, one by one (8191) 792
// (without rows ahead 1463).
template <typename T, int V, int W>
__global__ void __launch_bounds__(128, 5) k_sconv_fwd(ConvArgs a) {
  constexpr int K = W - 1, P = pairs_of<V>;
  __shared__ Vec<T, V> rows_ahead[V > 1 ? kDepth * 128 : 1];
  RowRing<T, ((V > 1) ? V : 4), kDepth, 128> ring(rows_ahead);
  const int c = ((int)(blockIdx.x % a.cblocks) * 128 + threadIdx.x) * V, tile_id = blockIdx.x / a.cblocks;
  if (c >= a.C) return;
  const T* x = static_cast<const T*>(a.x) + c;
  const T* s0 = a.s0 ? static_cast<const T*>(a.s0) + c : nullptr;
  T* out = static_cast<T*>(a.out) + c;
  T* st = a.st ? static_cast<T*>(a.st) + c : nullptr;
  uint64_t w[W][P], b[P], win[K][P];
  load_filters<T, V, W>(a, c, w, b);
  const int t0 = tile_id * a.tile, t1 = min(a.T, t0 + a.tile);
  auto end_state = [&](int d) {
    if (!st) return;
#pragma unroll
    for (int k = 0; k < K; ++k) store_pairs<T, V>(st + ((int64_t)d * K + k) * a.C, win[k]);
  };
  // The document the tile starts in; the empty documents at a position belong
  // to the tile that ends the token before them (position 0: to the first).
  int d = 0, t = t0;
  if (t0 == 0) {
    while (d < a.N && a.cu[d + 1] == 0) {
      load_window<T, V, W>(a, x, s0, d, 0, 0, win);
      end_state(d);
      ++d;
    }
  } else {
    d = doc_of(a.cu, a.N, t0);
  }
  while (t < t1) {
    const int ds = a.cu[d], de = a.cu[d + 1], e = min(de, t1);
    load_window<T, V, W>(a, x, s0, d, ds, t, win);
    auto token = [&](const Vec<T, V>& raw) {
      uint64_t xv[P], y[P];
      to_pairs<T, V>(raw, xv);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        uint64_t z = b[i];
#pragma unroll
        for (int k = 0; k < K; ++k) z = fma2(w[k][i], win[k][i], z);
        z = fma2(w[K][i], xv[i], z);
        if (a.silu) {
          float z0, z1;
          unpack2(z, z0, z1);
          z = mul2(z, pack2(sigmoid_f<T>(z0), V > 1 ? sigmoid_f<T>(z1) : 0.f));
        }
        y[i] = z;
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) win[k][i] = win[k + 1][i];
        win[K - 1][i] = xv[i];
      }
      store_pairs<T, V>(out + (int64_t)t * a.C, y);
    };
    if constexpr (V > 1) {
      const T* ahead = x + (int64_t)t * a.ldx;
      int tp = t;  // the next row to ask for
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {
        ring.push(i, ahead, tp < e);
        cp_async_commit();
        ahead += a.ldx;
        ++tp;
      }
#pragma unroll 1
      while (t < e) {
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
          if (t < e) {
            cp_async_wait<kDepth - 1>();
            token(ring.at(i));
            ring.push(i, ahead, tp < e);
            cp_async_commit();
            ahead += a.ldx;
            ++tp;
            ++t;
          }
        }
      }
      cp_async_wait<0>();
    } else {
      Vec<T, V> next[kDepth];
      auto fetch = [&](int from) {
#pragma unroll
        for (int i = 0; i < kDepth; ++i)
          if (from + i < e) next[i] = vload<T, V>(x + (int64_t)(from + i) * a.ldx);
      };
      fetch(t);
#pragma unroll 1
      while (t < e) {
        Vec<T, V> now[kDepth];
#pragma unroll
        for (int i = 0; i < kDepth; ++i) now[i] = next[i];
        fetch(t + kDepth);
#pragma unroll
        for (int i = 0; i < kDepth; ++i)
          if (t < e) {
            token(now[i]);
            ++t;
          }
      }
    }
    if (t == de) {
      end_state(d);
      ++d;
      while (d < a.N && a.cu[d + 1] == de) {
        load_window<T, V, W>(a, x, s0, d, de, de, win);
        end_state(d);
        ++d;
      }
    }
  }
}

struct ConvBwdArgs {
  ConvArgs f;
  const void* dout;
  int64_t ldo;
  const void* dst;  // [N][W-1][C] or null
  void *dx, *ds0;   // [T][C]; [N][W-1][C] or null
  float* part;      // [tiles][W + 1][C]: each tile's dw rows and dbias
};

// One thread owns V channels of one tile and walks it in token order: dz of
// token t completes dxx of row t - (W-1), whose partial sums are kept in W - 1
// registers a channel; dw and dbias accumulate in registers and leave as one
// partial row per tile.  The tile's last rows need dz of the W - 1 tokens after
// it, which are recomputed.  Bound by HBM (x and dout read, dx written) and by
// issue (66%): 32768 x 10240 in 396 us = 75% of the copy rate, 471 without rows ahead; 65536
// tokens x 8192 channels 619 us, 8190 763, 8191 1790.
template <typename T, int V, int W>
__global__ void __launch_bounds__(128, 5) k_sconv_bwd(ConvBwdArgs a) {
  constexpr int K = W - 1, P = pairs_of<V>;
  __shared__ Vec<T, V> rows_ahead[2][kRing<T, V> ? kDepth * 128 : 1];
  RowRing<T, (kRing<T, V> ? V : 4), kDepth, 128> rx_ring(rows_ahead[0]), rg_ring(rows_ahead[1]);
  const ConvArgs& f = a.f;
  const int c = ((int)(blockIdx.x % f.cblocks) * 128 + threadIdx.x) * V, tile_id = blockIdx.x / f.cblocks;
  if (c >= f.C) return;
  const T* x = static_cast<const T*>(f.x) + c;
  const T* dout = static_cast<const T*>(a.dout) + c;
  const T* s0 = f.s0 ? static_cast<const T*>(f.s0) + c : nullptr;
  const T* dst = a.dst ? static_cast<const T*>(a.dst) + c : nullptr;
  T* dx = static_cast<T*>(a.dx) + c;
  T* ds0 = a.ds0 ? static_cast<T*>(a.ds0) + c : nullptr;
  const uint64_t one = pack2(1.f, 1.f), minus = pack2(-1.f, -1.f);
  uint64_t w[W][P], b[P], win[K][P], acc[K][P], dw[W][P], db[P];
  load_filters<T, V, W>(f, c, w, b);
  zero_pairs<V>(db);
#pragma unroll
  for (int j = 0; j < W; ++j) zero_pairs<V>(dw[j]);
  const int t0 = tile_id * f.tile, t1 = min(f.T, t0 + f.tile);
  // The start state of an empty document is its end state.
  auto empty_doc = [&](int d) {
    if (!ds0) return;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      uint64_t g[P];
      if (dst) to_pairs<T, V>(vload<T, V>(dst + ((int64_t)d * K + k) * f.C), g);
      else zero_pairs<V>(g);
      store_pairs<T, V>(ds0 + ((int64_t)d * K + k) * f.C, g);
    }
  };
  int d = 0, t = t0;
  if (t0 == 0) {
    while (d < f.N && f.cu[d + 1] == 0) empty_doc(d++);
  } else {
    d = doc_of(f.cu, f.N, t0);
  }
  while (t < t1) {
    const int ds = f.cu[d], de = f.cu[d + 1];
    const bool fresh = t == ds;  // this tile owns the document's start-state rows
    const int e = min(de, t1);
    load_window<T, V, W>(f, x, s0, d, ds, t, win);
#pragma unroll
    for (int k = 0; k < K; ++k) zero_pairs<V>(acc[k]);
    const int own0 = fresh ? ds - K : t;  // rows [own0, t1) of this document are written here
    // dxx of row p is complete.
    auto emit = [&](int p, const uint64_t (&g)[P]) {
      if (p < own0 || p >= t1) return;
      if (p >= ds) store_pairs<T, V>(dx + (int64_t)p * f.C, g);
      else if (ds0) store_pairs<T, V>(ds0 + ((int64_t)d * K + (p - ds + K)) * f.C, g);
    };
    // Token tt: its dz, added to dw and dbias where the token is this tile's;
    // `done` gets dxx of row tt - K.
    auto token = [&](const Vec<T, V>& rx, const Vec<T, V>& rg, bool mine, uint64_t (&done)[P]) {
      uint64_t xv[P], g[P];
      to_pairs<T, V>(rx, xv);
      to_pairs<T, V>(rg, g);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        uint64_t dz = g[i];
        if (f.silu) {
          uint64_t z = b[i];
#pragma unroll
          for (int k = 0; k < K; ++k) z = fma2(w[k][i], win[k][i], z);
          z = fma2(w[K][i], xv[i], z);
          float z0, z1;
          unpack2(z, z0, z1);
          const uint64_t s = pack2(sigmoid_f<T>(z0), V > 1 ? sigmoid_f<T>(z1) : 0.f);
          // s + z s (1 - s)
          dz = mul2(dz, fma2(mul2(z, s), fma2(minus, s, one), s));
        }
        if (mine) {
          db[i] = add2(db[i], dz);
#pragma unroll
          for (int k = 0; k < K; ++k) dw[k][i] = fma2(dz, win[k][i], dw[k][i]);
          dw[K][i] = fma2(dz, xv[i], dw[K][i]);
        }
        // acc[k]: row tt - K + k
        done[i] = fma2(w[0][i], dz, acc[0][i]);
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) acc[k][i] = fma2(w[k + 1][i], dz, acc[k + 1][i]);
        acc[K - 1][i] = mul2(w[K][i], dz);
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) win[k][i] = win[k + 1][i];
        win[K - 1][i] = xv[i];
      }
    };
    auto rows = [&](int tt, Vec<T, V>& rx, Vec<T, V>& rg) {
      rx = vload<T, V>(x + (int64_t)tt * f.ldx);
      rg = vload<T, V>(dout + (int64_t)tt * a.ldo);
    };
    // the first K tokens, whose rows may be the start state's or another tile's
#pragma unroll 1
    for (int head = min(e, t + K); t < head; ++t) {
      Vec<T, V> rx, rg;
      uint64_t done[P];
      rows(t, rx, rg);
      token(rx, rg, true, done);
      emit(t - K, done);
    }
    if constexpr (kRing<T, V>) {
      const T *ax = x + (int64_t)t * f.ldx, *ag = dout + (int64_t)t * a.ldo;
      int tp = t;
      auto ask = [&](int i) {
        rx_ring.push(i, ax, tp < e);
        rg_ring.push(i, ag, tp < e);
        cp_async_commit();
        ax += f.ldx;
        ag += a.ldo;
        ++tp;
      };
#pragma unroll
      for (int i = 0; i < kDepth; ++i) ask(i);
      T* to = dx + (int64_t)(t - K) * f.C;
#pragma unroll 1
      while (t < e) {
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
          if (t < e) {
            cp_async_wait<kDepth - 1>();
            uint64_t done[P];
            token(rx_ring.at(i), rg_ring.at(i), true, done);
            ask(i);
            store_pairs<T, V>(to, done);
            to += f.C;
            ++t;
          }
        }
      }
      cp_async_wait<0>();
    }
    if constexpr (!kRing<T, V>) {
      constexpr int U = 4;
      Vec<T, V> nx[U], ng[U];
      auto fetch = [&](int from) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (from + i < e) rows(from + i, nx[i], ng[i]);
      };
      fetch(t);
      T* to = dx + (int64_t)(t - K) * f.C;
#pragma unroll 1
      while (t < e) {
        Vec<T, V> rx[U], rg[U];
#pragma unroll
        for (int i = 0; i < U; ++i) rx[i] = nx[i], rg[i] = ng[i];
        fetch(t + U);
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (t < e) {
            uint64_t done[P];
            token(rx[i], rg[i], true, done);
            store_pairs<T, V>(to, done);
            to += f.C;
            ++t;
          }
      }
    }
    // the rest, and the tokens after the tile that the tile's last rows feed
    const int tail = min(de, e + K);
#pragma unroll 1
    for (int tt = t; tt < tail; ++tt) {
      Vec<T, V> rx, rg;
      uint64_t done[P];
      rows(tt, rx, rg);
      token(rx, rg, tt < e, done);
      emit(tt - K, done);
    }
    t = e;
    if (tail == de) {  // the document's last rows: the end state's gradient joins
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (dst) {
          uint64_t g[P];
          to_pairs<T, V>(vload<T, V>(dst + ((int64_t)d * K + k) * f.C), g);
#pragma unroll
          for (int i = 0; i < P; ++i) acc[k][i] = add2(acc[k][i], g[i]);
        }
        emit(de - K + k, acc[k]);
      }
    }
    if (e == de) {
      ++d;
      while (d < f.N && f.cu[d + 1] == de) empty_doc(d++);
    }
  }
  next_may_start();  // (the sum of the partial rows)
  float* part = a.part + (int64_t)tile_id * (W + 1) * f.C + c;
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    float o[V + 1];
#pragma unroll
    for (int i = 0; i < P; ++i) unpack2(j < W ? dw[j < W ? j : 0][i] : db[i], o[2 * i], o[2 * i + 1]);
#pragma unroll
    for (int v = 0; v < V; ++v) part[(int64_t)j * f.C + v] = o[v];
  }
}

// dw[c][j] and dbias[c]: the tiles' partial rows summed in a fixed order (15 us for
// 10240 channels).
__global__ void __launch_bounds__(512) k_sconv_wgrad(const float* __restrict__ part, int tiles, int C, int W,
                                                     float* dw, float* db) {
  __shared__ float s[16][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, j = blockIdx.y;
  float sum = 0.f;
  previous_ended();
  if (c < C) {
#pragma unroll 8
    for (int i = row; i < tiles; i += 16) sum += part[((int64_t)i * (W + 1) + j) * C + c];
  }
  s[row][lane] = sum;
  __syncthreads();
  if (row == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 16; ++i) sum += s[i][lane];
    if (j < W) dw[(int64_t)c * W + j] = sum;
    else if (db) db[c] = sum;
  }
}

struct ConvStepArgs {
  const void *x, *weight, *bias;
  int wf32;
  int64_t ldx;
  void* state;        // [S][W-1][C]
  const int* slots;   // [B] or null
  int B, S, C;
  int silu;
  void* out;          // [B][C]
};

// One token of each sequence: the state's rows move up by one and x becomes
// its last.  Bound by the launch: 4 us a call of one sequence or a few.
template <typename T, int V, int W>
__global__ void __launch_bounds__(128) k_sconv_step(ConvStepArgs a) {
  constexpr int K = W - 1;
  const int c = (blockIdx.x * 128 + threadIdx.x) * V;
  if (c >= a.C) return;
  for (int i = blockIdx.y; i < a.B; i += gridDim.y) {
    const int slot = a.slots ? a.slots[i] : i;
    T* out = static_cast<T*>(a.out) + (int64_t)i * a.C + c;
    float y[V];
    if (slot < 0 || slot >= a.S) {  // an inactive row
#pragma unroll
      for (int v = 0; v < V; ++v) y[v] = 0.f;
      vstore<T, V>(out, y);
      continue;
    }
    T* st = static_cast<T*>(a.state) + (int64_t)slot * K * a.C + c;
    Vec<T, V> win[W];
#pragma unroll
    for (int k = 0; k < K; ++k) win[k] = vload<T, V>(st + (int64_t)k * a.C);
    win[K] = vload<T, V>(static_cast<const T*>(a.x) + (int64_t)i * a.ldx + c);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float z = a.bias ? load_param<T>(a.bias, a.wf32, c + v) : 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j)
        z = fmaf(load_param<T>(a.weight, a.wf32, (int64_t)(c + v) * W + j), to_f<T>(win[j].e[v]), z);
      y[v] = a.silu ? z * sigmoid_f<T>(z) : z;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) *reinterpret_cast<Vec<T, V>*>(st + (int64_t)k * a.C) = win[k + 1];
    vstore<T, V>(out, y);
  }
}

// Tokens a thread walks: about `most`, so that the rows read again at a tile's
// ends stay a small share, and such that the blocks fill whole waves of `wave`
// blocks (what the GPU holds at a time); short tiles only where there is too
// little to fill one.
int tile_tokens(int64_t T, int64_t cblocks, int wave, int most) {
  int64_t waves = (T * cblocks + (int64_t)wave * most - 1) / ((int64_t)wave * most);
  if (waves < 1) waves = 1;
  int64_t tiles = wave * waves / cblocks;
  if (tiles < 1) tiles = 1;
  int64_t tile = (T + tiles - 1) / tiles;
  if (tile < 16) tile = 16;
  return (int)tile;
}
// The partial rows a backward leaves do not depend on alignment, so that the
// workspace does not either: its tile is that of threads of eight bytes of BF16.
int bwd_tile_tokens(int64_t T, int64_t C) { return tile_tokens(T, ((C + 3) / 4 + 127) / 128, 152 * 5, 256); }

size_t elem(int dtype) { return dtype == GDR_DTYPE_F32 ? 4 : 2; }

// Runs f(type tag, vector width, taps) for the run-time type, alignment and W.
template <typename T, int V, typename F>
cudaError_t with_taps(int W, F f) {
  if (W == 2) return f(T(), std::integral_constant<int, V>(), std::integral_constant<int, 2>());
  if (W == 3) return f(T(), std::integral_constant<int, V>(), std::integral_constant<int, 3>());
  return f(T(), std::integral_constant<int, V>(), std::integral_constant<int, 4>());
}
template <int BYTES, typename F>
cudaError_t dispatch(int dtype, int V, int W, F f) {
  auto half = [&](auto t) {
    using T = decltype(t);
    return V > 2 ? with_taps<T, BYTES / 2>(W, f) : V == 2 ? with_taps<T, 2>(W, f) : with_taps<T, 1>(W, f);
  };
  switch (dtype) {
    case GDR_DTYPE_BF16: return half(__nv_bfloat16());
    case GDR_DTYPE_F16: return half(__half());
    default: return V > 1 ? with_taps<float, BYTES / 4>(W, f) : with_taps<float, 1>(W, f);
  }
}
// Channels a thread: BYTES of them where the channels, the rows' strides (or'ed into
// `strides`) and the addresses (`all`) allow it, else, of 16 bits, pairs, else one.
template <int BYTES>
int width(int dtype, int64_t C, int64_t strides, uintptr_t all) {
  const int e = (int)elem(dtype);
  for (int V = BYTES / e; V > 1; V = e == 2 && V > 2 ? 2 : 1)
    if (((C | strides) & (V - 1)) == 0 && (all & (uintptr_t)(V * e - 1)) == 0) return V;
  return 1;
}

gdr_status conv_check(int dtype, int wdtype, int64_t T, int64_t ldx, int32_t C, int32_t W, const void* x,
                      const void* weight) {
  if (dtype < 0 || dtype > GDR_DTYPE_F32 || (wdtype != dtype && wdtype != GDR_DTYPE_F32)) return GDR_INVALID_ARG;
  if (C <= 0 || W < 2 || W > 4 || T < 0 || (T > 1 && ldx < C)) return GDR_INVALID_ARG;
  if (T > GDR_OPS_MAX_T || C > GDR_OPS_MAX_T) return GDR_INVALID_ARG;  // a tile's or block's end stays an int
  if (T > 0 && (!x || !weight)) return GDR_INVALID_ARG;
  return GDR_OK;
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

gdr_status sconv_workspace_bytes(int64_t T, int32_t C, int32_t W, size_t* scratch_bytes) {
  if (!scratch_bytes || T < 0 || T > GDR_OPS_MAX_T || C <= 0 || C > GDR_OPS_MAX_T || W < 2 || W > 4) return GDR_INVALID_ARG;
  const int tile = bwd_tile_tokens(T, C);
  const int64_t tiles = T > 0 ? (T + tile - 1) / tile : 1;
  *scratch_bytes = (size_t)tiles * (W + 1) * C * sizeof(float);
  return GDR_OK;
}

gdr_status sconv_fwd(int dtype, const void* x, int64_t ldx, const void* weight, const void* bias, int wdtype,
                     const int32_t* cu_seqlens, const int32_t* cu_seqlens_host, int32_t N, int64_t T, int32_t C,
                     int32_t W, int silu, const void* s0, void* out, void* st, cudaStream_t stream) {
  gdr_status rc = conv_check(dtype, wdtype, T, ldx, C, W, x, weight);
  if (rc != GDR_OK) return rc;
  int64_t nc = 0;
  if ((rc = plan_host(T, N, cu_seqlens_host, &nc)) != GDR_OK) return rc;
  if (N == 0 || (T == 0 && !st)) return GDR_OK;
  if (!cu_seqlens || !weight || (T > 0 && !out)) return GDR_INVALID_ARG;
  // other tiles read rows of x and s0 after a tile has written its own
  if ((T > 0 && out == x) || (st && st == s0)) return GDR_INVALID_ARG;
  if ((rc = check_device()) != GDR_OK) return rc;
  ConvArgs a{x, weight, bias, wdtype == GDR_DTYPE_F32, ldx, cu_seqlens, N, (int)T, C, silu, s0, out, st, 0, 0};
  const int V = width<16>(dtype, C, ldx, (uintptr_t)x | (uintptr_t)out | (uintptr_t)s0 | (uintptr_t)st), nv = C / V;
  a.cblocks = (nv + 127) / 128;
  a.tile = tile_tokens(T, a.cblocks, 152 * 5, 128);
  const int64_t grid = (T > 0 ? (T + a.tile - 1) / a.tile : 1) * a.cblocks;
  if (grid > INT32_MAX) return GDR_INVALID_ARG;
  ProfScope ps("sconv_fwd", stream, (double)T * C);
  const cudaError_t e = dispatch<16>(dtype, V, W, [&](auto t, auto v, auto w) {
    k_sconv_fwd<decltype(t), decltype(v)::value, decltype(w)::value><<<(unsigned)grid, 128, 0, stream>>>(a);
    return cudaGetLastError();
  });
  return e == cudaSuccess ? GDR_OK : GDR_CUDA_ERROR;
}

gdr_status sconv_bwd(int dtype, const void* x, int64_t ldx, const void* weight, const void* bias, int wdtype,
                     const int32_t* cu_seqlens, const int32_t* cu_seqlens_host, int32_t N, int64_t T, int32_t C,
                     int32_t W, int silu, const void* s0, const void* dout, int64_t lddout, const void* dst, void* dx,
                     float* dweight, float* dbias, void* ds0, void* scratch, size_t scratch_bytes,
                     cudaStream_t stream) {
  gdr_status rc = conv_check(dtype, wdtype, T, ldx, C, W, x, weight);
  if (rc != GDR_OK) return rc;
  int64_t nc = 0;
  if ((rc = plan_host(T, N, cu_seqlens_host, &nc)) != GDR_OK) return rc;
  if (!weight || !dweight || !scratch || !cu_seqlens) return GDR_INVALID_ARG;
  if (T > 0 && (!dout || !dx || (T > 1 && lddout < C))) return GDR_INVALID_ARG;
  size_t need = 0;
  sconv_workspace_bytes(T, C, W, &need);
  if (((uintptr_t)scratch & 255) != 0) return GDR_INVALID_ARG;
  if (scratch_bytes < need) return GDR_WORKSPACE_TOO_SMALL;
  if ((T > 0 && (dx == x || dx == dout)) || (ds0 && (ds0 == dst || ds0 == s0))) return GDR_INVALID_ARG;
  if ((rc = check_device()) != GDR_OK) return rc;
  ConvBwdArgs a{};
  a.f = ConvArgs{x, weight, bias, wdtype == GDR_DTYPE_F32, ldx, cu_seqlens, N, (int)T, C, silu, s0, nullptr, nullptr,
                 0, 0};
  a.dout = dout;
  a.ldo = lddout;
  a.dst = dst;
  a.dx = dx;
  a.ds0 = ds0;
  a.part = static_cast<float*>(scratch);
  const uintptr_t all = (uintptr_t)x | (uintptr_t)s0 | (uintptr_t)dout | (uintptr_t)dst | (uintptr_t)dx | (uintptr_t)ds0;
  // 8 bytes a thread at most: the sums kept in registers are W of them a channel
  const int V = width<8>(dtype, C, ldx | lddout, all), nv = C / V;
  a.f.tile = bwd_tile_tokens(T, C);
  a.f.cblocks = (nv + 127) / 128;
  const int64_t tiles = T > 0 ? (T + a.f.tile - 1) / a.f.tile : 1, grid = tiles * a.f.cblocks;
  if (grid > INT32_MAX) return GDR_INVALID_ARG;
  {
    ProfScope ps("sconv_bwd", stream, (double)T * C);
    const cudaError_t e = dispatch<8>(dtype, V, W, [&](auto t, auto v, auto w) {
      k_sconv_bwd<decltype(t), decltype(v)::value, decltype(w)::value><<<(unsigned)grid, 128, 0, stream>>>(a);
      return cudaGetLastError();
    });
    if (e != cudaSuccess) return GDR_CUDA_ERROR;
  }
  ProfScope ps("sconv_wgrad", stream);
  return launch_early(k_sconv_wgrad, dim3((C + 31) / 32, W + 1), 512, 0, stream, a.part, (int)tiles, C, W, dweight, dbias) ==
                 cudaSuccess ? GDR_OK : GDR_CUDA_ERROR;
}

gdr_status sconv_step(int dtype, const void* x, int64_t ldx, const void* weight, const void* bias, int wdtype,
                      void* state, const int32_t* slots, int32_t B, int32_t S, int32_t C, int32_t W, int silu,
                      void* out, cudaStream_t stream) {
  gdr_status rc = conv_check(dtype, wdtype, B, ldx, C, W, x, weight);
  if (rc != GDR_OK) return rc;
  if (S < 0 || (!slots && B > S)) return GDR_INVALID_ARG;
  if (B == 0) return GDR_OK;
  if (!out || (S > 0 && !state)) return GDR_INVALID_ARG;
  if ((rc = check_device()) != GDR_OK) return rc;
  ConvStepArgs a{x, weight, bias, wdtype == GDR_DTYPE_F32, ldx, state, slots, B, S, C, silu, out};
  const int V = width<8>(dtype, C, ldx, (uintptr_t)x | (uintptr_t)state | (uintptr_t)out), nv = C / V;
  ProfScope ps("sconv_step", stream, (double)B * C);
  const cudaError_t e = dispatch<8>(dtype, V, W, [&](auto t, auto v, auto w) {
    k_sconv_step<decltype(t), decltype(v)::value, decltype(w)::value>
        <<<dim3((nv + 127) / 128, B < 65535 ? B : 65535), 128, 0, stream>>>(a);
    return cudaGetLastError();
  });
  return e == cudaSuccess ? GDR_OK : GDR_CUDA_ERROR;
}

}  // extern "C"
