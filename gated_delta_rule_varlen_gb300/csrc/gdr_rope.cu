// gdr_rope.cu -- rotary positions: the first R elements of every head of q and k in
// pairs (a, b), turned by the token's position times the pair's frequency,
//   (a, b) -> amplitude (a cos t - b sin t, b cos t + a sin t),  t = position frequency,
// the rest copied.  Pairs are elements (i, i + R / 2), or (2 i, 2 i + 1) interleaved.
// The gradient of the turned rows turns the other way.
//
// The angle keeps its accuracy at far positions without 64-bit floating point: the
// frequency in turns a token is a 64-bit binary fraction, whose product with the
// position, modulo 2^64, is the angle's fraction of a turn, and the top 32 bits of it become
// sine and cosine.  The fraction of a token is off by (1 + f / 260) 2^-64 turns: what is cut off,
// and the rounding of 2^66 / (2 pi) to 64 bits.  Frequencies that are not finite turn to NaN.
//
// Bound by HBM: each element read once and written once; 32768 tokens of 40 heads of 128 in
// BF16 take 121 us, 82% of the copy rate (FP32 96%).  A block turns the heads of some
// tokens; their sines and cosines are formed once, into shared memory (by every thread for
// its own columns, over several heads, 175 us).
#include <algorithm>

#include "gdr_ops.cuh"
#include "gdr_runtime.h"

namespace gdr {
namespace {

struct RopeRows {
  const void* x;
  int64_t s0, s1;  // element strides of a token and of a head
  void* y;
  int64_t y0, y1;
};
struct RopeArgs {
  RopeRows q, k;
  int HQ, H;           // query heads; with the key heads
  int D, R;
  int64_t T;
  const void* pos;     // or null: counted from each document's start
  int pos64;
  const int* cu;
  int N;
  const float* freq;   // [R / 2]
  float amp;
  int back;
  int units, turned;   // pieces of a head: all, those that turn
  int tokens;          // of a block
  int copy;            // where the second piece of a unit to copy lies (0: it has none)
};

constexpr int THREADS = 256;
// Most elements of a token: a thread's count of units passes their number by a step of the loop.
constexpr int64_t ROPE_MAX_ROW = INT32_MAX - 16 * THREADS;
// Units a thread asks for together: of eight elements (two pieces of 16 bytes each) two, so
// that an SM holds four blocks (64 registers a thread); with four of them it held two.
constexpr int rope_ahead(int V) { return V == 8 ? 2 : 4; }

// 2^64 of the fraction of a turn that frequency f (radians) advances: f = m 2^(e - 150)
// times 1 / (2 pi) = kTurn 2^-66, in integers (64-bit floating point has 1/64 of their rate).
constexpr unsigned long long kTurn = 0xa2f9836e4e44152aull;
__device__ __forceinline__ uint64_t turns_of(float f) {
  const uint32_t bits = __float_as_uint(f) & 0x7fffffffu, ex = bits >> 23;
  const uint64_t m = ex ? (bits & 0x7fffffu) | 0x800000u : bits;
  const uint64_t lo = m * kTurn, hi = __umul64hi(m, kTurn);
  const int sh = 152 - (ex ? (int)ex : 1);  // product 2^-sh
  uint64_t u;
  if (sh >= 64) u = sh < 128 ? hi >> (sh - 64) : 0;
  else if (sh > 0) u = lo >> sh | hi << (64 - sh);
  else u = sh > -64 ? lo << -sh : 0;
  return f < 0.f ? 0 - u : u;
}
__device__ __forceinline__ void angle(float f, uint64_t pos, float amp, bool back, float& c, float& s) {
  const int top = (int)((turns_of(f) * pos) >> 32);  // [-1/2, 1/2) turns
  sincospif((float)top * 4.656612873077393e-10f, &s, &c);
  if (!(fabsf(f) < INFINITY)) c = s = NAN;
  c *= amp;
  s *= back ? -amp : amp;
}

// A unit of a head: V elements from each half of the turned part (interleaved: of V / 2 pairs
// each), or V elements of the rest to copy (from each half of it where its size allows).
// LOOSE: rows on no common boundary, element by element; interleaved one pair a unit.
template <typename T, int V, bool LOOSE>
__device__ __forceinline__ Vec<T, V> load_piece(const T* p, int n) {
  if constexpr (!LOOSE) return vload<T, V>(p);
  Vec<T, V> v{};
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < n) v.e[i] = p[i];
  return v;
}
template <typename T, int V, bool LOOSE>
__device__ __forceinline__ void store_piece(T* p, const Vec<T, V>& v, int n) {
  if constexpr (!LOOSE) {
    *reinterpret_cast<Vec<T, V>*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = v.e[i];
  }
}
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> packed(const float (&f)[V]) {
  Vec<T, V> v;
#pragma unroll
  for (int i = 0; i < V; ++i) v.e[i] = from_f<T>(f[i]);
  return v;
}

template <typename T, int V, bool INTER, bool LOOSE>
__global__ void __launch_bounds__(THREADS, 4) k_rope(const __grid_constant__ RopeArgs a) {
  constexpr bool TWO = !(INTER && LOOSE);  // pieces of a turned unit
  constexpr int PAIRS = INTER ? V / 2 : V, U = rope_ahead(V);  // units asked for together
  extern __shared__ __align__(16) float rope_smem[];
  const int half = a.R / 2;
  float *cs = rope_smem, *sn = rope_smem + a.tokens * half;  // [tokens][R / 2]
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int tokens = (int)min((int64_t)a.tokens, a.T - t0);
  // The next U units of the thread: unit, head and token advance by sums with carries.
  const int per = a.units * a.H, n = tokens * per;
  const int du = THREADS % a.units, dh = THREADS / a.units % a.H, dt = THREADS / per;
  int u = threadIdx.x % a.units, h = threadIdx.x / a.units % a.H, t = threadIdx.x / per;
  struct Unit {
    const T* x;
    T* y;
    int u, t;
    Vec<T, V> lo, hi;
  };
  auto load = [&](Unit& w) {
    w.u = u;
    w.t = t;
    const bool isq = h < a.HQ, turn = u < a.turned;
    const RopeRows& r = isq ? a.q : a.k;
    const int hh = isq ? h : h - a.HQ, c0 = turn ? u * V : a.R + (u - a.turned) * V;
    w.x = static_cast<const T*>(r.x) + (t0 + t) * r.s0 + hh * r.s1 + c0;
    w.y = static_cast<T*>(r.y) + (t0 + t) * r.y0 + hh * r.y1 + c0;
    w.lo = load_piece<T, V, LOOSE>(w.x, a.D - c0);
    if (turn ? TWO : a.copy > 0) w.hi = load_piece<T, V, LOOSE>(w.x + (turn ? half : a.copy), V);
    u += du;
    const int cu = u >= a.units;
    u -= cu ? a.units : 0;
    h += dh + cu;
    const int ch = h >= a.H;
    h -= ch ? a.H : 0;
    t += dt + ch;
  };
  Unit w[U];
  int i = threadIdx.x;
  previous_ended();
#pragma unroll
  for (int j = 0; j < U; ++j)
    if (i + j * THREADS < n) load(w[j]);  // (on their way while the angles are formed)
  for (int e = threadIdx.x; e < tokens * half; e += THREADS) {
    const int64_t at = t0 + e / half;
    uint64_t pos;
    if (!a.pos) pos = (uint64_t)(at - a.cu[doc_of(a.cu, a.N, (int)at)]);
    else if (a.pos64) pos = (uint64_t)static_cast<const int64_t*>(a.pos)[at];
    else pos = (uint64_t)(int64_t)static_cast<const int*>(a.pos)[at];
    angle(__ldg(a.freq + e % half), pos, a.amp, a.back, cs[e], sn[e]);
  }
  __syncthreads();
  while (i < n) {
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (i + j * THREADS < n) {
        const Unit& k = w[j];
        if (k.u >= a.turned) {
          store_piece<T, V, LOOSE>(k.y, k.lo, a.D - (a.R + (k.u - a.turned) * V));
          if (a.copy > 0) store_piece<T, V, LOOSE>(k.y + a.copy, k.hi, V);
          continue;
        }
        // PAIRS sines and cosines from pair `at` on
        auto angles = [&](int at, float (&c)[PAIRS], float (&s)[PAIRS]) {
          if (PAIRS % 4 == 0 && half % 8 == 0) {
#pragma unroll
            for (int e = 0; e < PAIRS; e += 4) {
              const float4 x = *reinterpret_cast<const float4*>(cs + at + e), y = *reinterpret_cast<const float4*>(sn + at + e);
              c[e] = x.x, c[(e + 1) % PAIRS] = x.y, c[(e + 2) % PAIRS] = x.z, c[(e + 3) % PAIRS] = x.w;
              s[e] = y.x, s[(e + 1) % PAIRS] = y.y, s[(e + 2) % PAIRS] = y.z, s[(e + 3) % PAIRS] = y.w;
            }
          } else {
#pragma unroll
            for (int e = 0; e < PAIRS; ++e) c[e] = cs[at + e], s[e] = sn[at + e];
          }
        };
        float c[PAIRS], s[PAIRS], f[V], g[V];
        const int at = k.t * half + k.u * PAIRS;
        angles(at, c, s);
        vunpack<T, V>(k.lo, f);
        if constexpr (INTER) {
          auto turn = [&](float (&v)[V]) {
#pragma unroll
            for (int e = 0; e < PAIRS; ++e) {
              const float p = v[2 * e], q = v[2 * e + 1];
              v[2 * e] = p * c[e] - q * s[e];
              v[2 * e + 1] = q * c[e] + p * s[e];
            }
          };
          turn(f);
          store_piece<T, V, LOOSE>(k.y, packed<T, V>(f), V);
          if constexpr (TWO) {
            angles(at + half / 2, c, s);
            vunpack<T, V>(k.hi, g);
            turn(g);
            store_piece<T, V, LOOSE>(k.y + half, packed<T, V>(g), V);
          }
        } else {
          vunpack<T, V>(k.hi, g);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float p = f[e], q = g[e];
            f[e] = p * c[e] - q * s[e];
            g[e] = q * c[e] + p * s[e];
          }
          store_piece<T, V, LOOSE>(k.y, packed<T, V>(f), V);
          store_piece<T, V, LOOSE>(k.y + half, packed<T, V>(g), V);
        }
      }
    i += U * THREADS;
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (i + j * THREADS < n) load(w[j]);
  }
}

// The widest pieces that every row allows: up to 16 bytes; 0: pairs side by side whose halves
// are no whole pieces of pairs.
int piece_of(const RopeArgs& a, int elem, bool inter) {
  for (int v = 16 / elem; v > 1; v /= 2) {
    bool ok = a.R / 2 % v == 0 && (a.D - a.R) % v == 0;
    for (const RopeRows* r : {&a.q, &a.k}) {
      if (r == &a.k && a.H == a.HQ) continue;
      const uintptr_t p = (uintptr_t)r->x | (uintptr_t)r->y;
      ok = ok && p % (v * elem) == 0 && r->s0 % v == 0 && r->s1 % v == 0 && r->y0 % v == 0 && r->y1 % v == 0;
    }
    if (ok) return v;
  }
  return inter ? 0 : 1;
}

template <typename T, int V, bool INTER, bool LOOSE = false>
cudaError_t launch(RopeArgs a, cudaStream_t st) {
  const int rest = a.D - a.R;
  a.turned = (INTER && LOOSE ? a.R : a.R / 2) / V;
  a.copy = rest > 0 && rest / 2 % V == 0 && rest % 2 == 0 ? rest / 2 : 0;
  a.units = a.turned + ((a.copy ? a.copy : rest) + V - 1) / V;
  // Tokens of a block: eight units a thread, which share the sines; sines up to 32 KB; fewer
  // where that leaves SMs without blocks (957 tokens of 8 heads of 64: 12.4 us with 15 blocks).
  const int64_t per = (int64_t)a.units * a.H;
  int64_t n = std::max<int64_t>(1, 8 * THREADS / per);
  if (a.R > 0) n = std::min<int64_t>(n, std::max(1, 4096 / (a.R / 2)));
  n = std::min<int64_t>(n, (a.T + 4 * sm_count() - 1) / (4 * sm_count()));
  a.tokens = (int)n;
  const int64_t blocks = (a.T + a.tokens - 1) / a.tokens;
  return launch_early(k_rope<T, V, INTER, LOOSE>, dim3((unsigned)blocks), THREADS, (size_t)a.tokens * a.R * sizeof(float), st, a);
}

template <typename T>
cudaError_t launch_t(const RopeArgs& a, bool inter, cudaStream_t st) {
  const int v = piece_of(a, sizeof(T), inter);
  if constexpr (sizeof(T) == 2)
    if (v == 8) return inter ? launch<T, 8, true>(a, st) : launch<T, 8, false>(a, st);
  if (v == 4) return inter ? launch<T, 4, true>(a, st) : launch<T, 4, false>(a, st);
  if (v == 2) return inter ? launch<T, 2, true>(a, st) : launch<T, 2, false>(a, st);
  return inter ? launch<T, 2, true, true>(a, st) : launch<T, 1, false>(a, st);
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" gdr_status rope_turn(gdr_dtype dtype, const void* q, int64_t qs0, int64_t qs1, int32_t HQ, void* q_out,
                                int64_t qo0, int64_t qo1, const void* k, int64_t ks0, int64_t ks1, int32_t HK, void* k_out,
                           int64_t ko0, int64_t ko1, int64_t T, int32_t D, int32_t R, const float* freqs,
                           const void* positions, int positions64, const int32_t* cu_seqlens, int32_t N,
                           int interleaved, float amplitude, int inverse, cudaStream_t stream) {
  if (dtype < 0 || dtype > GDR_DTYPE_F32 || T < 0 || T > GDR_OPS_MAX_T || HQ < 0 || HK < 0) return GDR_INVALID_ARG;
  if (D <= 0 || R < 0 || R > D || R > GDR_ROPE_MAX_R || R % 2 != 0 || (int64_t)D * ((int64_t)HQ + HK) > ROPE_MAX_ROW) return GDR_INVALID_ARG;
  if (T == 0 || HQ + HK == 0) return GDR_OK;
  if ((HQ > 0 && (!q || !q_out)) || (HK > 0 && (!k || !k_out)) || (R > 0 && !freqs)) return GDR_INVALID_ARG;
  if (R > 0 && !positions && (!cu_seqlens || N <= 0)) return GDR_INVALID_ARG;
  if (HQ > 0 && HK > 0 && (q_out == k_out || q_out == k || k_out == q)) return GDR_INVALID_ARG;
  const gdr_status rc = check_device();
  if (rc != GDR_OK) return rc;
  RopeArgs a{};
  a.q = {q, qs0, qs1, q_out, qo0, qo1};
  a.k = {k, ks0, ks1, k_out, ko0, ko1};
  a.HQ = HQ;
  a.H = HQ + HK;
  a.D = D;
  a.R = R;
  a.T = T;
  a.pos = positions;
  a.pos64 = positions64;
  a.cu = cu_seqlens;
  a.N = N;
  a.freq = freqs;
  a.amp = amplitude;
  a.back = inverse != 0;
  ProfScope ps("rope", stream, (double)T * a.H);
  const bool inter = interleaved != 0;
  const cudaError_t e = dtype == GDR_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, inter, stream)
                        : dtype == GDR_DTYPE_F16 ? launch_t<__half>(a, inter, stream)
                                                 : launch_t<float>(a, inter, stream);
  return e == cudaSuccess ? GDR_OK : GDR_CUDA_ERROR;
}
