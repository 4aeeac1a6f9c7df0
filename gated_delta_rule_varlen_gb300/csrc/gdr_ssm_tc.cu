// gdr_ssm_tc.cu -- the selective state space scan of prompts on the tensor
// cores, in chunks of Q = 128 tokens that restart at each document.
//
// Inside a chunk with start state S0 [N][P], gates a_t = dt_t A, prefix sums
// G_i = sum_{k<=i} a_k:
//   out_i = exp(G_i) C_i S0 + sum_{j<=i} M_ij x_j + D x_i,
//           M_ij = (C_i . B_j) exp(G_i - G_j) dt_j
//   S_end = exp(G_last) S0 + B^T (w x),  w_j = dt_j exp(sum_{k>j} a_k)
// Four products of 128-row tiles (tcgen05, FP32 accumulators in TMEM):
//   CB = C B^T,  Yo = C S0,  Yd = M x,  U = B^T (w x).
// x, B and C are BF16 and enter exactly; what is formed in FP32 (M, S0, w x)
// enters as a pair of BF16 numbers hi + lo (17 bits: FP32 end states within a
// few 1e-6, and the outputs' error stays that of their own rounding).  The state
// itself stays in FP32 registers.
//
// exp(G_i - G_j) is formed per 32-column block of M: for rows below the block
// as exp(G_i - G_r) exp(G_r - G_j) with r the block's last token (both factors
// at most 1, so neither overflows, and one that underflows belongs to a product
// that does), inside the diagonal block directly.
//
// A chunk's tiles land by TMA; rows past the document's end are cleared, since
// they hold another document's values (a NaN there would pass through a zero
// weight).  Within a document a non-finite value reaches the outputs of its
// whole chunk.
#include <algorithm>
#include <cudaTypedefs.h>

#include "gdr_ssm.cuh"
#include "gdr_tc.cuh"

namespace gdr {
namespace {

constexpr int Q = 128;        // tokens of a chunk
constexpr int PT = 64;        // columns of the state that a block works on
constexpr int BLK = Q * 128;  // bytes of a tile block: 128 rows of 64 BF16

struct TcArgs {
  CUtensorMap x_map, b_map, c_map;
  SsmArgs a;
  int pblocks;      // ceil(P / 64)
  int lseg;         // chunks of a segment at most
  float* seg;       // [segments][H][NS][P]: start states of split documents' segments
  float* gsum;      // [segments][H]: log2 decay over each segment
  int* err;
};

// The segment `idx` of document `doc`, its chunks [c0, c1) and tokens.
struct Seg {
  int doc, idx, nseg, tok0, len;  // first token and tokens of the segment
  int first;                      // the document's first segment
};

// Finds segment `want` by a scan over the documents (one warp).
__device__ Seg find_segment(const int* __restrict__ cu, int N, int lseg, int want) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int d0 = 0; d0 < N; d0 += 32) {
    const int d = d0 + lane;
    int n = 0, start = 0, len = 0;
    if (d < N) {
      start = cu[d];
      len = cu[d + 1] - start;
      const int ch = (len + Q - 1) / Q;
      n = ch == 0 ? 1 : (ch + lseg - 1) / lseg;
    }
    int pre = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, pre, m);
      if (lane >= m) pre += v;
    }
    const int total = __shfl_sync(0xffffffffu, pre, 31);
    if (want < base + total) {
      const unsigned hit = __ballot_sync(0xffffffffu, want < base + pre);
      const int l = __ffs(hit) - 1;
      Seg s;
      s.doc = d0 + l;
      s.nseg = __shfl_sync(0xffffffffu, n, l);
      s.first = base + __shfl_sync(0xffffffffu, pre, l) - s.nseg;
      s.idx = want - s.first;
      const int dl = __shfl_sync(0xffffffffu, len, l), ds = __shfl_sync(0xffffffffu, start, l);
      const int ch = (dl + Q - 1) / Q, per = ch / s.nseg, extra = ch % s.nseg;
      // the first `extra` segments have one chunk more
      const int c0 = s.idx * per + min(s.idx, extra), c1 = c0 + per + (s.idx < extra ? 1 : 0);
      s.tok0 = ds + c0 * Q;
      s.len = min(dl, c1 * Q) - c0 * Q;
      return s;
    }
    base += total;
  }
  return Seg{0, 0, 1, 0, 0, 0};
}

// Bounded wait that also gives up once another role of the block has.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  if (tc::mbar_try(bar, parity)) return true;
  const uint64_t t0 = tc::global_ns();
  while (!tc::mbar_try(bar, parity)) {
    if (*abort) return false;
    if (tc::global_ns() - t0 > 2000000000ull) {
      *abort = 1;
      atomicExch(err, 10);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(tc::smem_u32(bar)) : "memory");
}

constexpr uint32_t kIdescTransposeA = 1u << 15;

// Byte of the 16-byte piece c (8 BF16) of row r of a 128-byte-swizzled block.
__device__ __forceinline__ uint32_t piece(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// Two FP32 numbers as BF16 pairs: hi rounded to nearest, lo the rest rounded
// (off by at most 2^-18 of the number).
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  const __nv_bfloat162 l = __floats2bfloat162_rn(a - bf_lo(hi), b - bf_hi(hi));
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// Inclusive warp scan.
__device__ __forceinline__ float scan_up(float v, int lane) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const float u = __shfl_up_sync(0xffffffffu, v, m);
    if (lane >= m) v += u;
  }
  return v;
}
__device__ __forceinline__ float scan_down(float v, int lane) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const float u = __shfl_down_sync(0xffffffffu, v, m);
    if (lane + m < 32) v += u;
  }
  return v;
}

// Lane l loads the raw dt of tokens 4 l .. 4 l + 3 (zero past `len`: no step at all).
__device__ __forceinline__ void load_gates(const SsmArgs& a, int h, int tok0, int len, float (&dt)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = 4 * lane + i;
    dt[i] = j < len ? load_dt(a, tok0 + j, h) : 0.f;
  }
}

// Row j of a tile block to zero.
__device__ __forceinline__ void clear_row(unsigned char* tile, int j) {
#pragma unroll
  for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(tile + j * 128 + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
}

// xw rows: w_j x_j of token row j as hi and lo blocks.
__device__ __forceinline__ void build_xw(const unsigned char* x, unsigned char* hi, unsigned char* lo, int j, float w) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint4 v = *reinterpret_cast<const uint4*>(x + piece(j, c));
    uint4 h, l;
    split2(bf_lo(v.x) * w, bf_hi(v.x) * w, h.x, l.x);
    split2(bf_lo(v.y) * w, bf_hi(v.y) * w, h.y, l.y);
    split2(bf_lo(v.z) * w, bf_hi(v.z) * w, h.z, l.z);
    split2(bf_lo(v.w) * w, bf_hi(v.w) * w, h.w, l.w);
    *reinterpret_cast<uint4*>(hi + piece(j, c)) = h;
    *reinterpret_cast<uint4*>(lo + piece(j, c)) = l;
  }
}

// ---------------------------------------------------------------------------
// The walk: one block per (segment, head, 64 columns of the state).
//   warp 0: TMA;  warp 1: MMA issue, TMEM;  warp 2: gates
//   warps 4-7: M from CB;  warps 8-11: w x, the state;  warps 12-15: outputs
// Every role runs through the chunks on its own; barriers hand buffers over.
// ---------------------------------------------------------------------------
constexpr int WALK_THREADS = 512;
constexpr uint32_t T_CB = 0, T_YO = 128, T_YD = 192, T_U = 256, T_MH = 320, T_ML = 384;

struct WalkSmem {
  unsigned char B[2][2 * BLK], C[2][2 * BLK], X[2][BLK];
  unsigned char xw[2][BLK];  // hi, lo
  unsigned char S[2][BLK];   // hi, lo
  // One chunk's gates.  gc is read until the chunk's outputs leave, the others
  // only up to M and w x: single buffers (shared memory is full).
  float gc[2][Q];  // prefix sums of dt A log2(e)
  float dt[Q];
  float colf[Q];   // dt_j 2^(gc[end of j's 32-block] - gc_j)
  float w[Q];      // dt_j 2^(sum after j)
  float gam;       // 2^gc[last]
  uint64_t full[2], empty[2], gates[2], w_full;
  uint64_t cb_full, m_full, xw_full, u_full, s_full, y_full, y_empty, done;
  uint32_t tmem;
  int abort;
  Seg seg;
};

__global__ void __launch_bounds__(WALK_THREADS, 1) k_ssm_walk(const __grid_constant__ TcArgs ta) {
  extern __shared__ __align__(1024) unsigned char ssm_smem[];  // tiles are swizzled in 1024-byte atoms
  WalkSmem& s = *reinterpret_cast<WalkSmem*>(ssm_smem);
  const SsmArgs& a = ta.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = a.H * ta.pblocks;
  const int hp = blockIdx.x % per, h = hp / ta.pblocks, p0 = (hp % ta.pblocks) * PT, sid = blockIdx.x / per;
  const int grp = h / (a.H / a.G);
  const int nblk = a.NS > 64 ? 2 : 1, ksteps = (a.NS + 15) / 16;
  if (warp == 0) {
    const Seg sg = find_segment(a.cu, a.N, ta.lseg, sid);
    if (lane == 0) {
      s.seg = sg;
      s.abort = 0;
      for (int i = 0; i < 2; ++i) {
        tc::mbar_init(&s.full[i], 1);
        tc::mbar_init(&s.empty[i], 1 + 128);
        tc::mbar_init(&s.gates[i], 32);
      }
      tc::mbar_init(&s.w_full, 32);
      tc::mbar_init(&s.cb_full, 1);
      tc::mbar_init(&s.m_full, 128);
      tc::mbar_init(&s.xw_full, 128);
      tc::mbar_init(&s.u_full, 1);
      tc::mbar_init(&s.s_full, 128);
      tc::mbar_init(&s.y_full, 1);
      tc::mbar_init(&s.y_empty, 128);
      tc::mbar_init(&s.done, 1);
      tc::mbar_fence_init();
    }
  }
  if (warp == 1) {
    tc::tmem_alloc(&s.tmem, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const Seg sg = s.seg;
  const uint32_t tmem = s.tmem;
  const int nch = (sg.len + Q - 1) / Q;
  const bool last_seg = sg.idx == sg.nseg - 1;
  volatile int* ab = &s.abort;
  int* err = ta.err;

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      for (int c = 0; c < nch; ++c) {
        const int b = c & 1;
        if (c >= 2 && !wait_or_abort(&s.empty[b], ((c >> 1) - 1) & 1, ab, err)) break;
        const int row = sg.tok0 + c * Q;
        tc::mbar_arrive_expect_tx(&s.full[b], (uint32_t)((1 + 2 * nblk) * BLK));
        for (int k = 0; k < nblk; ++k) {
          tc::tma_load_3d(s.C[b] + k * BLK, &ta.c_map, 64 * k, grp, row, &s.full[b]);
          tc::tma_load_3d(s.B[b] + k * BLK, &ta.b_map, 64 * k, grp, row, &s.full[b]);
        }
        tc::tma_load_3d(s.X[b], &ta.x_map, p0, h, row, &s.full[b]);
        issued = c + 1;
      }
      // no copy is in flight when the block ends
      for (int c = max(0, issued - 2); c < issued; ++c) tc::mbar_wait(&s.full[c & 1], (c >> 1) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t i_cb = tc::idesc_bf16(128, 128);
      constexpr uint32_t i_yo = tc::idesc_bf16(128, PT) | tc::kIdescTransposeB;
      constexpr uint32_t i_u = i_yo | kIdescTransposeA;
      bool ok = true;
      auto cb = [&](int c) {  // CB = C B^T
        const int b = c & 1;
        ok = ok && wait_or_abort(&s.full[b], (c >> 1) & 1, ab, err);
        if (!ok) return;
        tc::tc_fence_after();
        const uint64_t dc = tc::desc_k_sw128(s.C[b]), db = tc::desc_k_sw128(s.B[b]);
        for (int k = 0; k < ksteps; ++k)
          tc::mma_bf16(tmem + T_CB, tc::kstep32(dc, k, Q), tc::kstep32(db, k, Q), i_cb, k > 0);
        tc::mma_commit(&s.cb_full);
      };
      if (nch > 0) cb(0);
      for (int c = 0; c < nch && ok; ++c) {
        const int b = c & 1;
        // U = B^T (w x): the previous U has been read once w x of this chunk is there
        ok = ok && wait_or_abort(&s.xw_full, c & 1, ab, err);
        if (!ok) break;
        tc::tc_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t da = tc::desc_mn_sw128(s.B[b] + k * 2048, BLK, 1024);
          tc::mma_bf16(tmem + T_U, da, tc::desc_mn_sw128(s.xw[0] + k * 2048, BLK, 1024), i_u, k > 0);
          tc::mma_bf16(tmem + T_U, da, tc::desc_mn_sw128(s.xw[1] + k * 2048, BLK, 1024), i_u, 1);
        }
        tc::mma_commit(&s.u_full);
        // Yo = C S0
        ok = ok && wait_or_abort(&s.s_full, c & 1, ab, err);
        if (c > 0) ok = ok && wait_or_abort(&s.y_empty, (c - 1) & 1, ab, err);
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t dc = tc::desc_k_sw128(s.C[b]);
        for (int k = 0; k < ksteps; ++k) {
          tc::mma_bf16(tmem + T_YO, tc::kstep32(dc, k, Q), tc::desc_mn_sw128(s.S[0] + k * 2048, BLK, 1024), i_yo, k > 0);
          tc::mma_bf16(tmem + T_YO, tc::kstep32(dc, k, Q), tc::desc_mn_sw128(s.S[1] + k * 2048, BLK, 1024), i_yo, 1);
        }
        // Yd = M x
        ok = ok && wait_or_abort(&s.m_full, c & 1, ab, err);
        if (!ok) break;
        tc::tc_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t dx = tc::desc_mn_sw128(s.X[b] + k * 2048, BLK, 1024);
          tc::mma_f16_ta(tmem + T_YD, tmem + T_MH + 8 * k, dx, i_yo, k > 0);
          tc::mma_f16_ta(tmem + T_YD, tmem + T_ML + 8 * k, dx, i_yo, 1);
        }
        tc::mma_commit(&s.y_full);
        tc::mma_commit(&s.empty[b]);
        if (c + 1 < nch) cb(c + 1);
      }
      // no MMA is in flight when the block ends
      if (nch > 0) {
        tc::mma_commit(&s.done);
        tc::mbar_wait(&s.done, 0);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    float dt[4], nx[4];
    if (nch > 0) load_gates(a, h, sg.tok0, min(Q, sg.len), nx);
    const float A = a.A[h] * LOG2E;
    for (int c = 0; c < nch; ++c) {
      const int b = c & 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) dt[i] = nx[i];
      if (c + 1 < nch) load_gates(a, h, sg.tok0 + (c + 1) * Q, min(Q, sg.len - (c + 1) * Q), nx);
      float g[4], r[4];  // inclusive prefix; exclusive suffix (summed from the end, where it is small)
      float run = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        run = fmaf(dt[i], A, run);
        g[i] = run;
      }
      float before = __shfl_up_sync(0xffffffffu, scan_up(run, lane), 1);
      float after = __shfl_down_sync(0xffffffffu, scan_down(run, lane), 1);
      if (lane == 0) before = 0.f;
      if (lane == 31) after = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] += before;
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        r[i] = after;
        after = fmaf(dt[i], A, after);
      }
      const float blk_end = __shfl_sync(0xffffffffu, g[3], lane | 7);
      const float4 w = make_float4(dt[0] * exp2f(r[0]), dt[1] * exp2f(r[1]), dt[2] * exp2f(r[2]), dt[3] * exp2f(r[3]));
      const float4 cf = make_float4(dt[0] * exp2f(blk_end - g[0]), dt[1] * exp2f(blk_end - g[1]),
                                    dt[2] * exp2f(blk_end - g[2]), dt[3] * exp2f(blk_end - g[3]));
      bool ok = c == 0 || wait_or_abort(&s.xw_full, (c - 1) & 1, ab, err);
      if (!__all_sync(0xffffffffu, ok)) break;
      *reinterpret_cast<float4*>(&s.w[4 * lane]) = w;
      if (lane == 31) s.gam = exp2f(g[3]);
      arrive(&s.w_full);
      ok = c == 0 || wait_or_abort(&s.m_full, (c - 1) & 1, ab, err);
      if (c >= 2) ok = ok && wait_or_abort(&s.empty[b], ((c >> 1) - 1) & 1, ab, err);
      if (!__all_sync(0xffffffffu, ok)) break;
      *reinterpret_cast<float4*>(&s.gc[b][4 * lane]) = make_float4(g[0], g[1], g[2], g[3]);
      *reinterpret_cast<float4*>(&s.dt[4 * lane]) = make_float4(dt[0], dt[1], dt[2], dt[3]);
      *reinterpret_cast<float4*>(&s.colf[4 * lane]) = cf;
      arrive(&s.gates[b]);
    }
  } else if (warp >= 4 && warp < 8) {
    // M: thread = row i; column blocks b < w by factors, b == w directly, b > w zero
    const int w = warp - 4, i = 32 * w + lane;
    const uint32_t row = tmem + ((uint32_t)(32 * w) << 16);
    {
      uint32_t z[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) z[q] = 0u;
      for (int b = w + 1; b < 4; ++b) {
        tc::tmem_st16(row + T_MH + 16 * b, z);
        tc::tmem_st16(row + T_ML + 16 * b, z);
      }
      tc::tmem_wait_st();
    }
    for (int c = 0; c < nch; ++c) {
      const int st = c & 1;
      bool ok = wait_or_abort(&s.gates[st], (c >> 1) & 1, ab, err) && wait_or_abort(&s.cb_full, c & 1, ab, err);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc::tc_fence_after();
      const float* gc = s.gc[st];
      const float gi = gc[i];
      for (int b = 0; b <= w; ++b) {
        uint32_t v[32], hi[16], lo[16];
        tc::tmem_ld32(row + T_CB + 32 * b, v);
        const float rf = ex2(gi - gc[32 * b + 31]);
        tc::tmem_wait_ld();
        if (b < w) {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 cf = *reinterpret_cast<const float4*>(&s.colf[32 * b + j]);
            split2(__uint_as_float(v[j]) * (cf.x * rf), __uint_as_float(v[j + 1]) * (cf.y * rf), hi[j / 2], lo[j / 2]);
            split2(__uint_as_float(v[j + 2]) * (cf.z * rf), __uint_as_float(v[j + 3]) * (cf.w * rf), hi[j / 2 + 1],
                   lo[j / 2 + 1]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 gj = *reinterpret_cast<const float2*>(&gc[32 * b + j]);
            const float2 dj = *reinterpret_cast<const float2*>(&s.dt[32 * b + j]);
            const float m0 = j <= lane ? __uint_as_float(v[j]) * (dj.x * ex2(gi - gj.x)) : 0.f;
            const float m1 = j + 1 <= lane ? __uint_as_float(v[j + 1]) * (dj.y * ex2(gi - gj.y)) : 0.f;
            split2(m0, m1, hi[j / 2], lo[j / 2]);
          }
        }
        // the previous chunk's Yd has read M
        if (b == 0 && c > 0) {
          ok = wait_or_abort(&s.y_full, (c - 1) & 1, ab, err);
          tc::tc_fence_after();
        }
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc::tmem_st16(row + T_MH + 16 * b, hi);
        tc::tmem_st16(row + T_ML + 16 * b, lo);
      }
      if (!ok) break;
      tc::tmem_wait_st();
      tc::tc_fence_before();
      arrive(&s.m_full);
    }
  } else if (warp >= 8 && warp < 12) {
    // w x of token row j, and state row n (both 32 (warp - 8) + lane)
    const int j = tid - 256, n = j;
    const uint32_t row = tmem + ((uint32_t)(32 * (warp - 8)) << 16);
    float S[PT];
    const float* start = nullptr;
    if (sg.idx > 0) start = ta.seg + (((int64_t)sid * a.H + h) * a.NS + n) * a.P + p0;
    else if (a.h0) start = a.h0 + (((int64_t)sg.doc * a.H + h) * a.NS + n) * a.P + p0;
#pragma unroll
    for (int p = 0; p < PT; p += 4) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (start && n < a.NS && p0 + p < a.P) v = *reinterpret_cast<const float4*>(start + p);
      S[p] = v.x;
      S[p + 1] = v.y;
      S[p + 2] = v.z;
      S[p + 3] = v.w;
    }
    float gam = 0.f;
    bool ok = true;
    auto advance = [&](int c) {  // S = gam S + U of chunk c
      ok = ok && wait_or_abort(&s.u_full, c & 1, ab, err);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      tc::tc_fence_after();
#pragma unroll
      for (int p = 0; p < PT; p += 32) {
        uint32_t u[32];
        tc::tmem_ld32(row + T_U + p, u);
        tc::tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 32; ++q) S[p + q] = fmaf(gam, S[p + q], __uint_as_float(u[q]));
      }
      tc::tc_fence_before();
    };
    for (int c = 0; c < nch; ++c) {
      const int b = c & 1, len = min(Q, sg.len - c * Q);
      if (c > 0) advance(c - 1);
      ok = ok && wait_or_abort(&s.full[b], (c >> 1) & 1, ab, err);
      ok = ok && wait_or_abort(&s.w_full, c & 1, ab, err);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (j >= len) {
        clear_row(s.X[b], j);
        for (int k = 0; k < nblk; ++k) clear_row(s.B[b] + k * BLK, j);
      }
      gam = s.gam;
      build_xw(s.X[b], s.xw[0], s.xw[1], j, s.w[j]);
      tc::fence_proxy_async();
      arrive(&s.xw_full);
      // S0 as operand, once the previous chunk's Yo has read the old one
      if (c > 0) ok = wait_or_abort(&s.y_full, (c - 1) & 1, ab, err);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        uint4 hi, lo;
        split2(S[8 * q], S[8 * q + 1], hi.x, lo.x);
        split2(S[8 * q + 2], S[8 * q + 3], hi.y, lo.y);
        split2(S[8 * q + 4], S[8 * q + 5], hi.z, lo.z);
        split2(S[8 * q + 6], S[8 * q + 7], hi.w, lo.w);
        *reinterpret_cast<uint4*>(s.S[0] + piece(n, q)) = hi;
        *reinterpret_cast<uint4*>(s.S[1] + piece(n, q)) = lo;
      }
      tc::fence_proxy_async();
      arrive(&s.s_full);
    }
    if (ok && nch > 0) advance(nch - 1);
    if (ok && last_seg && a.ht && n < a.NS) {
      float* to = a.ht + (((int64_t)sg.doc * a.H + h) * a.NS + n) * a.P + p0;
#pragma unroll
      for (int p = 0; p < PT; p += 4)
        if (p0 + p < a.P) *reinterpret_cast<float4*>(to + p) = make_float4(S[p], S[p + 1], S[p + 2], S[p + 3]);
    }
  } else if (warp >= 12) {
    // outputs of token row i
    const int w = warp - 12, i = 32 * w + lane;
    const uint32_t row = tmem + ((uint32_t)(32 * w) << 16);
    const float D = a.D ? a.D[h] : 0.f;
    for (int c = 0; c < nch; ++c) {
      const int b = c & 1, len = min(Q, sg.len - c * Q);
      bool ok = wait_or_abort(&s.full[b], (c >> 1) & 1, ab, err);
      ok = ok && wait_or_abort(&s.gates[b], (c >> 1) & 1, ab, err);
      ok = ok && wait_or_abort(&s.y_full, c & 1, ab, err);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc::tc_fence_after();
      const float e = ex2(s.gc[b][i]);
      __nv_bfloat16* out = a.out + ((int64_t)(sg.tok0 + c * Q + i) * a.H + h) * a.P + p0;
#pragma unroll
      for (int p = 0; p < PT; p += 32) {
        uint32_t yo[32], yd[32];
        tc::tmem_ld32(row + T_YO + p, yo);
        tc::tmem_ld32(row + T_YD + p, yd);
        tc::tmem_wait_ld();
        if (p + 32 == PT) {
          tc::tc_fence_before();
          arrive(&s.y_empty);
        }
#pragma unroll
        for (int q = 0; q < 32; q += 8) {
          const uint4 xv = *reinterpret_cast<const uint4*>(s.X[b] + piece(i, (p + q) / 8));
          const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
          uint32_t o[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int k = q + 2 * z;
            const float y0 = fmaf(D, bf_lo(xs[z]), fmaf(e, __uint_as_float(yo[k]), __uint_as_float(yd[k])));
            const float y1 = fmaf(D, bf_hi(xs[z]), fmaf(e, __uint_as_float(yo[k + 1]), __uint_as_float(yd[k + 1])));
            const __nv_bfloat162 y = __floats2bfloat162_rn(y0, y1);
            o[z] = *reinterpret_cast<const uint32_t*>(&y);
          }
          if (i < len && p0 + p + q < a.P)
            *reinterpret_cast<uint4*>(out + p + q) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      arrive(&s.empty[b]);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Summary of a segment (split documents only): its end state from a zero start,
//   U = B^T (w x) with w_j = dt_j exp(sum of the gates after j in the segment),
// accumulated in TMEM over its chunks, last chunk first, and its total decay.
//   warp 0: TMA;  warp 1: MMA;  warp 2: gates;  warps 4-7 / 8-11: w x of the
//   even / odd steps
// ---------------------------------------------------------------------------
constexpr int SUM_THREADS = 384;
struct SumSmem {
  unsigned char B[2][2 * BLK], X[2][BLK];
  unsigned char xw[2][2][BLK];  // step parity; hi, lo
  float w[2][Q];
  uint64_t full[2], empty[2], gates[2], xw_full[2], done;
  uint32_t tmem;
  int abort;
  Seg seg;
};

__global__ void __launch_bounds__(SUM_THREADS, 1) k_ssm_sum(const __grid_constant__ TcArgs ta) {
  extern __shared__ __align__(1024) unsigned char ssm_smem[];
  SumSmem& s = *reinterpret_cast<SumSmem*>(ssm_smem);
  const SsmArgs& a = ta.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = a.H * ta.pblocks;
  const int hp = blockIdx.x % per, h = hp / ta.pblocks, p0 = (hp % ta.pblocks) * PT, sid = blockIdx.x / per;
  const int grp = h / (a.H / a.G);
  const int nblk = a.NS > 64 ? 2 : 1;
  if (warp == 0) {
    const Seg sg = find_segment(a.cu, a.N, ta.lseg, sid);
    if (lane == 0) {
      s.seg = sg;
      s.abort = 0;
      for (int i = 0; i < 2; ++i) {
        tc::mbar_init(&s.full[i], 1);
        tc::mbar_init(&s.empty[i], 1);
        tc::mbar_init(&s.gates[i], 32);
        tc::mbar_init(&s.xw_full[i], 128);
      }
      tc::mbar_init(&s.done, 1);
      tc::mbar_fence_init();
    }
  }
  __syncthreads();
  const Seg sg = s.seg;
  if (sg.idx == sg.nseg - 1) return;  // no segment starts from this one's end
  if (warp == 1) {
    tc::tmem_alloc(&s.tmem, 64);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s.tmem;
  const int nch = sg.len / Q;  // a segment that is not its document's last holds whole chunks
  volatile int* ab = &s.abort;
  int* err = ta.err;

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      for (int k = 0; k < nch; ++k) {
        const int b = k & 1, row = sg.tok0 + (nch - 1 - k) * Q;
        if (k >= 2 && !wait_or_abort(&s.empty[b], ((k >> 1) - 1) & 1, ab, err)) break;
        tc::mbar_arrive_expect_tx(&s.full[b], (uint32_t)((1 + nblk) * BLK));
        for (int q = 0; q < nblk; ++q) tc::tma_load_3d(s.B[b] + q * BLK, &ta.b_map, 64 * q, grp, row, &s.full[b]);
        tc::tma_load_3d(s.X[b], &ta.x_map, p0, h, row, &s.full[b]);
        issued = k + 1;
      }
      for (int k = max(0, issued - 2); k < issued; ++k) tc::mbar_wait(&s.full[k & 1], (k >> 1) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t i_u = tc::idesc_bf16(128, PT) | tc::kIdescTransposeB | kIdescTransposeA;
      for (int k = 0; k < nch; ++k) {
        const int b = k & 1;
        if (!wait_or_abort(&s.xw_full[b], (k >> 1) & 1, ab, err)) break;
        tc::tc_fence_after();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint64_t da = tc::desc_mn_sw128(s.B[b] + q * 2048, BLK, 1024);
          tc::mma_bf16(tmem, da, tc::desc_mn_sw128(s.xw[b][0] + q * 2048, BLK, 1024), i_u, k + q > 0);
          tc::mma_bf16(tmem, da, tc::desc_mn_sw128(s.xw[b][1] + q * 2048, BLK, 1024), i_u, 1);
        }
        tc::mma_commit(&s.empty[b]);
      }
      tc::mma_commit(&s.done);
      tc::mbar_wait(&s.done, 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    const float A = a.A[h] * LOG2E;
    float tail = 0.f, dt[4], nx[4];  // the gates after this chunk
    if (nch > 0) load_gates(a, h, sg.tok0 + (nch - 1) * Q, Q, nx);
    for (int k = 0; k < nch; ++k) {
      const int b = k & 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) dt[i] = nx[i];
      if (k + 1 < nch) load_gates(a, h, sg.tok0 + (nch - 2 - k) * Q, Q, nx);
      const bool ok = k < 2 || wait_or_abort(&s.empty[b], ((k >> 1) - 1) & 1, ab, err);
      if (!__all_sync(0xffffffffu, ok)) break;
      const float run = ((dt[0] + dt[1]) + (dt[2] + dt[3])) * A;
      const float inc = scan_down(run, lane);
      float after = __shfl_down_sync(0xffffffffu, inc, 1);
      after = (lane == 31 ? 0.f : after) + tail;
      float4 v;
      v.w = dt[3] * exp2f(after);
      after = fmaf(dt[3], A, after);
      v.z = dt[2] * exp2f(after);
      after = fmaf(dt[2], A, after);
      v.y = dt[1] * exp2f(after);
      after = fmaf(dt[1], A, after);
      v.x = dt[0] * exp2f(after);
      *reinterpret_cast<float4*>(&s.w[b][4 * lane]) = v;
      tail += __shfl_sync(0xffffffffu, inc, 0);
      arrive(&s.gates[b]);
    }
    if (lane == 0 && p0 == 0) ta.gsum[(int64_t)sid * a.H + h] = tail;
  } else if (warp >= 4) {
    const int g = (warp - 4) >> 2, j = (tid - 128) & 127;
    for (int k = g; k < nch; k += 2) {
      bool ok = wait_or_abort(&s.full[g], (k >> 1) & 1, ab, err);
      ok = ok && wait_or_abort(&s.gates[g], (k >> 1) & 1, ab, err);
      if (k >= 2) ok = ok && wait_or_abort(&s.empty[g], ((k >> 1) - 1) & 1, ab, err);
      if (!ok) break;
      build_xw(s.X[g], s.xw[g][0], s.xw[g][1], j, s.w[g][j]);
      tc::fence_proxy_async();
      arrive(&s.xw_full[g]);
    }
  }
  __syncthreads();
  tc::tc_fence_after();
  if (warp >= 4 && warp < 8 && !s.abort) {
    const int n = tid - 128;
    const uint32_t row = tmem + ((uint32_t)(32 * (warp - 4)) << 16);
    float* to = ta.seg + (((int64_t)sid * a.H + h) * a.NS + n) * a.P + p0;
#pragma unroll
    for (int p = 0; p < PT; p += 32) {
      uint32_t u[32];
      tc::tmem_ld32(row + p, u);
      tc::tmem_wait_ld();
      if (n < a.NS) {
#pragma unroll
        for (int q = 0; q < 32; q += 4)
          if (p0 + p + q < a.P) *reinterpret_cast<uint4*>(to + p + q) = make_uint4(u[q], u[q + 1], u[q + 2], u[q + 3]);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(tmem, 64);
}

// The start states of split documents' segments, in place of the segments' own
// end states: S[s + 1] = 2^gsum[s] S[s] + U[s].  One thread per state element.
__global__ void __launch_bounds__(256) k_ssm_merge(const __grid_constant__ TcArgs ta) {
  const SsmArgs& a = ta.a;
  const int64_t elems = (int64_t)a.NS * a.P;
  const int eblocks = (int)((elems + 1023) / 1024);
  const int e0 = (blockIdx.x % eblocks) * 1024 + threadIdx.x * 4, h = (blockIdx.x / eblocks) % a.H;
  const int d = blockIdx.x / eblocks / a.H;
  // the document's first segment: the segments of the documents before it
  int before = 0;
  for (int i = threadIdx.x; i < d; i += 256) {
    const int ch = (a.cu[i + 1] - a.cu[i] + Q - 1) / Q;
    before += ch == 0 ? 1 : (ch + ta.lseg - 1) / ta.lseg;
  }
  __shared__ int sums[8];
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) before += __shfl_xor_sync(0xffffffffu, before, m);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = before;
  __syncthreads();
  before = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) before += sums[i];
  const int ch = (a.cu[d + 1] - a.cu[d] + Q - 1) / Q, nseg = ch == 0 ? 1 : (ch + ta.lseg - 1) / ta.lseg;
  if (nseg == 1 || e0 >= elems) return;
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.h0) S = *reinterpret_cast<const float4*>(a.h0 + ((int64_t)d * a.H + h) * elems + e0);
  const int64_t step = (int64_t)a.H * elems;
  float* at = ta.seg + ((int64_t)before * a.H + h) * elems + e0;
  const float* gs = ta.gsum + (int64_t)before * a.H + h;
  for (int s0 = 0; s0 < nseg; s0 += 8) {
    float4 u[8];
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s0 + i < nseg - 1) {
        u[i] = *reinterpret_cast<const float4*>(at + (s0 + i) * step);
        g[i] = exp2f(gs[(int64_t)(s0 + i) * a.H]);
      }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s0 + i < nseg) {
        *reinterpret_cast<float4*>(at + (s0 + i) * step) = S;
        if (s0 + i < nseg - 1) {
          S.x = fmaf(g[i], S.x, u[i].x);
          S.y = fmaf(g[i], S.y, u[i].y);
          S.z = fmaf(g[i], S.z, u[i].z);
          S.w = fmaf(g[i], S.w, u[i].w);
        }
      }
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// [T][heads][dim] BF16, tokens ld elements apart, one head at a time: boxes of
// 64 elements x 1 head x 128 tokens, 128-byte swizzle, zero fill outside.
bool token_map(CUtensorMap* map, const void* base, uint64_t T, uint64_t heads, uint64_t dim, uint64_t ld) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {dim, heads, T};
  cuuint64_t strides[2] = {dim * 2, ld * 2};
  cuuint32_t box[3] = {64, 1, Q};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

bool ssm_tc_shape(int P, int NS) { return P % 8 == 0 && NS % 8 == 0 && NS <= 128; }

bool ssm_tc_layout(const SsmArgs& a) {
  const uintptr_t all = (uintptr_t)a.x | (uintptr_t)a.B | (uintptr_t)a.C | (uintptr_t)a.out | (uintptr_t)a.h0 |
                        (uintptr_t)a.ht;
  if ((all & 15) != 0) return false;
  return a.T <= 1 || (a.ldx % 8 == 0 && a.ldb % 8 == 0 && a.ldc % 8 == 0);
}

// Whole documents while they keep the SMs evenly busy; else the segment length
// with the least estimated time, in chunk steps of one block: kStart steps to
// start a block, kSum for a summary's step.
SsmPlan ssm_tc_plan(int H, int P, int NS, int N, const int32_t* cu) {
  constexpr double kStart = 3.0, kSum = 0.4;
  const int64_t items = (int64_t)H * ((P + 63) / 64);
  const double sms = 152.0;
  int64_t nc = 0, most = 0;
  for (int i = 0; i < N; ++i) {
    const int64_t ch = (cu[i + 1] - (int64_t)cu[i] + Q - 1) / Q;
    nc += ch;
    most = std::max(most, ch);
  }
  SsmPlan best{(int)std::max<int64_t>(most, 1), N, false, 0};
  double cost = std::max((double)(nc + kStart * N) * items / sms, most + kStart);
  // pieces of the longest document
  for (int64_t k = 2; k <= 256 && (most + k - 1) / k >= 4; ++k) {
    const int64_t L = (most + k - 1) / k;
    int64_t nseg = 0, again = 0;
    for (int i = 0; i < N; ++i) {
      const int64_t ch = (cu[i + 1] - (int64_t)cu[i] + Q - 1) / Q;
      const int64_t n = ch == 0 ? 1 : (ch + L - 1) / L;
      nseg += n;
      if (n > 1) again += ch - ch / n;
    }
    const double waves = (double)nseg * items / sms;
    const double walk = std::max((nc + kStart * nseg) * items / sms, (double)(L + kStart) * (int64_t)(waves + 0.999));
    const double sum = std::max(kSum * again * items / sms, kSum * L) + 2 * kStart;
    if (walk + sum < 0.95 * cost) {
      cost = walk + sum;
      best.lseg = (int)L;
      best.nseg = nseg;
      best.split = true;
    }
  }
  if (best.split)
    best.scratch = up256((size_t)best.nseg * H * NS * P * sizeof(float)) + up256((size_t)best.nseg * H * sizeof(float));
  return best;
}

cudaError_t launch_ssm_tc(const SsmArgs& a, const SsmPlan& plan, void* scratch, cudaStream_t st) {
  TcArgs t{};
  t.a = a;
  t.pblocks = (a.P + 63) / 64;
  t.lseg = plan.lseg;
  t.err = device_error_ptr();
  if (!t.err) return cudaErrorUnknown;
  if (a.T > 0) {
    const uint64_t one = 8;  // a single token's stride is never used
    if (!token_map(&t.x_map, a.x, a.T, a.H, a.P, a.T > 1 ? a.ldx : (uint64_t)a.H * a.P * one) ||
        !token_map(&t.b_map, a.B, a.T, a.G, a.NS, a.T > 1 ? a.ldb : (uint64_t)a.G * a.NS * one) ||
        !token_map(&t.c_map, a.C, a.T, a.G, a.NS, a.T > 1 ? a.ldc : (uint64_t)a.G * a.NS * one))
      return cudaErrorInvalidValue;
  }
  const unsigned grid = (unsigned)(plan.nseg * a.H * t.pblocks);
  constexpr int sm_walk = (int)sizeof(WalkSmem), sm_sum = (int)sizeof(SumSmem);
  static_assert(sm_walk <= 232448 && sm_sum <= 232448, "227 KB of shared memory a block");
  if (plan.split) {
    t.seg = static_cast<float*>(scratch);
    t.gsum = reinterpret_cast<float*>(static_cast<char*>(scratch) +
                                      up256((size_t)plan.nseg * a.H * a.NS * a.P * sizeof(float)));
    cudaFuncSetAttribute(k_ssm_sum, cudaFuncAttributeMaxDynamicSharedMemorySize, sm_sum);
    {
      ProfScope ps("ssm_sum", st, (double)a.T * a.H);
      k_ssm_sum<<<grid, SUM_THREADS, sm_sum, st>>>(t);
    }
    if (cudaError_t e = cudaGetLastError()) return e;
    ProfScope ps("ssm_merge", st);
    const unsigned mb = (unsigned)(((int64_t)a.NS * a.P + 1023) / 1024) * a.H * a.N;
    k_ssm_merge<<<mb, 256, 0, st>>>(t);
    if (cudaError_t e = cudaGetLastError()) return e;
  }
  cudaFuncSetAttribute(k_ssm_walk, cudaFuncAttributeMaxDynamicSharedMemorySize, sm_walk);
  ProfScope ps("ssm_walk", st, (double)a.T * a.H);
  k_ssm_walk<<<grid, WALK_THREADS, sm_walk, st>>>(t);
  return cudaGetLastError();
}

}  // namespace gdr
