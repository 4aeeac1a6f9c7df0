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
// x, B and C are BF16 and enter exactly.  w x enters U as the sum of three BF16
// numbers (24 bits), so that the state, kept in FP32 registers from chunk to
// chunk, is that of FP32 arithmetic.  M and S0, which only outputs depend on, enter
// as pairs of BF16 numbers: a term of an output's sums is off by at most 2^-17 of
// itself, so that the output's own rounding (2^-9) is what is left of it unless
// the terms cancel to some 2^-8 of their size.  (One BF16 number each is not
// enough: the error is 2^-9 of |C| |S|, not of the output, 4e-2 of it where the state's
// rows share a large part that C is orthogonal to.)
//
// exp(G_i - G_j) is formed from the difference, at most 1 on and below the
// diagonal; what is above is dropped by selection.
//
// A chunk's tiles land by TMA; rows past the document's end are cleared, since
// they hold another document's values (a NaN there would pass through a zero
// weight).  Within a document a non-finite value reaches the outputs of its
// whole chunk.
#include <cudaTypedefs.h>

#include <algorithm>
#include <functional>
#include <new>
#include <utility>
#include <vector>

#include "gdr_ssm.cuh"
#include "gdr_tc.cuh"

namespace gdr {
namespace {

constexpr int Q = 128;        // tokens of a chunk
constexpr int PT = 64;        // columns of the state that a block works on
constexpr int BLK = Q * 128;  // bytes of a tile block: 128 rows of 64 BF16
constexpr int GATES = 2 * Q + 96;  // floats of a chunk's gates

struct TcArgs {
  CUtensorMap x_map, b_map, c_map, out_map;
  SsmArgs a;
  const float* gates;  // [chunks][H][GATES], written by k_ssm_gates (Gates)
  int pblocks;      // ceil(P / 64)
  int pairs;        // summaries: two neighbours a block
  int lseg;         // chunks of a segment at most
  float* seg;       // [split documents' segments][H][NS][P]: their start states
  float* gsum;      // [split documents' segments][H]: log2 decay over each
  int* err;
};

// The segment `idx` of document `doc`, its chunks [c0, c1) and tokens.
struct Seg {
  int doc, idx, nseg, tok0, len;  // first token and tokens of the segment
  int chunk0;                     // its first chunk; an empty document counts as one
  int slot;                       // its place among the segments of split documents
};

// A token's gate dt A (log2).  Below -128 it is -128: ex2 of either is zero (it flushes
// below 2^-126), while a chunk's prefix sums stay above -2^14, where the differences
// that the decays between other tokens are formed from keep 2^-11; of sums that a
// reset of -1e9 had entered nothing would be left.  (A NaN stays.)
__device__ __forceinline__ float gate_log2(float dt, float A) {
  float a;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(dt * A), "f"(-128.f));
  return a;
}

// A chunk's gates of one head (a_t = gate_log2(dt_t, A log2 e)):
//   ss[j]   sum of the a after token j: 2^(ss_j - ss_i) is the decay from j to i,
//           and dt_j 2^ss_j = w_j keeps its accuracy, since ss is summed from the end
//   dt[j]   activated (zero past the document's end)
//   colf[j] dt_j 2^(ss_j - ss[end of j's 32 tokens]), j < 96
struct Gates {
  const float* p;
  __device__ __forceinline__ const float* ss() const { return p; }
  __device__ __forceinline__ const float* dt() const { return p + Q; }
  __device__ __forceinline__ const float* colf() const { return p + 2 * Q; }
  // the chunk's whole decay (log2; the first token's gate as it is: below -128 all of it is zero)
  __device__ __forceinline__ float total(float A) const { return fmaf(*dt(), A, *ss()); }
};
__device__ __forceinline__ Gates gates_of(const TcArgs& t, int chunk, int h) {
  return Gates{t.gates + ((int64_t)chunk * t.a.H + h) * GATES};
}

// Finds segment `want` by a scan over the documents (one warp).
__device__ Seg find_segment(const int* __restrict__ cu, int N, int lseg, int want) {
  const int lane = threadIdx.x & 31;
  int base = 0, cbase = 0, whole = 0;  // documents that are not split
#pragma unroll 1
  for (int d0 = 0; d0 < N; d0 += 32) {
    const int d = d0 + lane;
    int n = 0, start = 0, len = 0, nc = 0;
    if (d < N) {
      start = cu[d];
      len = cu[d + 1] - start;
      const int ch = (len + Q - 1) / Q;
      n = ch == 0 ? 1 : (ch + lseg - 1) / lseg;
      nc = ch == 0 ? 1 : ch;
    }
    int pre = n, cpre = nc;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, pre, m), w = __shfl_up_sync(0xffffffffu, cpre, m);
      if (lane >= m) {
        pre += v;
        cpre += w;
      }
    }
    const int total = __shfl_sync(0xffffffffu, pre, 31), ctotal = __shfl_sync(0xffffffffu, cpre, 31);
    const unsigned ones = __ballot_sync(0xffffffffu, n == 1);
    if (want < base + total) {
      const unsigned hit = __ballot_sync(0xffffffffu, want < base + pre);
      const int l = __ffs(hit) - 1;
      Seg s;
      s.doc = d0 + l;
      s.nseg = __shfl_sync(0xffffffffu, n, l);
      s.idx = want - (base + __shfl_sync(0xffffffffu, pre, l) - s.nseg);
      const int dl = __shfl_sync(0xffffffffu, len, l), ds = __shfl_sync(0xffffffffu, start, l);
      const int ch = (dl + Q - 1) / Q, per = ch / s.nseg, extra = ch % s.nseg;
      // the first `extra` segments have one chunk more
      const int c0 = s.idx * per + min(s.idx, extra), c1 = c0 + per + (s.idx < extra ? 1 : 0);
      s.tok0 = ds + c0 * Q;
      s.len = min(dl, c1 * Q) - c0 * Q;
      s.chunk0 = cbase + __shfl_sync(0xffffffffu, cpre - nc, l) + c0;
      s.slot = want - whole - __popc(ones & ((1u << l) - 1));
      return s;
    }
    base += total;
    cbase += ctotal;
    whole += __popc(ones);
  }
  return Seg{0, 0, 1, 0, 0, 0, 0};
}

// Waits of the blocks' roles.  Each gives up after kTries tries of at most a
// microsecond, or once another role has, and returns false; the block then
// reports the timeout as it ends.  Few instructions: the roles run straight
// through long loops that share the instruction cache.
constexpr int kTries = 1 << 20;
__device__ __forceinline__ bool try_phase(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(tc::smem_u32(bar)), "r"(parity), "r"(1000u)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort) {
  for (int tries = 0; !try_phase(bar, parity); ++tries)
    if (tries > kTries || *abort) {
      *abort = 1;
      return false;
    }
  return true;
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(tc::smem_u32(bar)) : "memory");
}

constexpr uint32_t kIdescTransposeA = 1u << 15;

// Byte of the 16-byte piece c (8 BF16) of row r of a 128-byte-swizzled block.
__device__ __forceinline__ uint32_t piece(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// The two BF16 of a word as a pair of FP32.
__device__ __forceinline__ uint64_t widen2(uint32_t w) { return pack2(bf_lo(w), bf_hi(w)); }

// A pair of FP32 numbers rounded to BF16.
__device__ __forceinline__ uint32_t round2(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// What rounding them leaves of a pair of FP32 numbers, rounded to BF16: the two
// together hold 17 bits of each (the rest's sign is one).
__device__ __forceinline__ uint32_t rest2(uint64_t v) { return round2(fma2(widen2(round2(v)), pack2(-1.f, -1.f), v)); }
__device__ __forceinline__ void split2(uint64_t v, uint32_t& hi, uint32_t& lo) {
  hi = round2(v);
  lo = round2(fma2(widen2(hi), pack2(-1.f, -1.f), v));
}
// A pair of FP32 numbers as three BF16 pairs, each the rest of the ones before it
// rounded: all 24 bits.
__device__ __forceinline__ void split3(uint64_t v, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  const uint64_t minus = pack2(-1.f, -1.f);
  hi = round2(v);
  v = fma2(widen2(hi), minus, v);
  mid = round2(v);
  lo = round2(fma2(widen2(mid), minus, v));
}

// Shared-memory matrix descriptors of 128-byte-swizzled tiles share their upper
// word (8-row groups 1024 bytes apart, descriptor version 1, the swizzle); the
// lower word is the address in 16-byte units and, for MN-major tiles, the
// distance of the 64-element blocks along MN.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(const void* tile) { return tc::smem_u32(tile) >> 4 | (BLK / 16) << 16; }

// MMAs and commits that a whole warp walks through together and one elected
// thread performs (the same one each time).  Measured: 36 clocks an MMA of 64
// columns from TMEM and 53 from shared memory, its read time; picked by a
// comparison of the lane instead, 72 for either.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 da, db;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 db;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 db, {%2, %5};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(tc::smem_u32(bar))
      : "memory");
}
// The same values, known to be the same on every lane: what is computed from
// them (loop bounds, operand addresses) can live in uniform registers.
__device__ __forceinline__ Seg uniform(const Seg& s) {
  Seg u;
  u.doc = __shfl_sync(0xffffffffu, s.doc, 0);
  u.idx = __shfl_sync(0xffffffffu, s.idx, 0);
  u.nseg = __shfl_sync(0xffffffffu, s.nseg, 0);
  u.tok0 = __shfl_sync(0xffffffffu, s.tok0, 0);
  u.len = __shfl_sync(0xffffffffu, s.len, 0);
  u.chunk0 = __shfl_sync(0xffffffffu, s.chunk0, 0);
  u.slot = __shfl_sync(0xffffffffu, s.slot, 0);
  return u;
}
// One arrival for the warp, after all its lanes' work.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive(bar);
}
// The wait of a whole warp: the same answer on every lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  for (int tries = 0; !__all_sync(0xffffffffu, try_phase(bar, parity)); ++tries)
    if (__any_sync(0xffffffffu, tries > kTries || *abort)) {
      *abort = 1;
      return false;
    }
  return true;
}
// tcgen05.wait::ld with the loaded registers as operands: nothing that reads
// them can be scheduled before it.
__device__ __forceinline__ void wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void wait_ld(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
// Eight consecutive TMEM columns of the warp's lanes to registers (complete
// after wait_ld).
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ uint64_t pair_of(const uint32_t* r) {
  return pack2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
// ---------------------------------------------------------------------------
// The gates of every chunk: one block per (chunk, 32 heads).  dt is read with
// the heads on the lanes (its rows are tokens), then each warp scans whole
// heads, four tokens a lane.
// ---------------------------------------------------------------------------
constexpr int GATE_WARPS = 16;
__global__ void __launch_bounds__(GATE_WARPS * 32) k_ssm_gates(const int* __restrict__ cu, SsmArgs a, float* gates) {
  __shared__ float sdt[Q][33];
  __shared__ Seg sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  next_may_start();
  if (warp == 0) {
    const Seg sg = find_segment(cu, a.N, 1, blockIdx.x);
    if (lane == 0) sh = sg;
  }
  __syncthreads();
  const Seg sg = sh;
  const int h0 = blockIdx.y * 32, h = h0 + lane;
  const float bias = h < a.H && a.dt_bias ? a.dt_bias[h] : 0.f;
  float v[Q / GATE_WARPS];  // all rows asked for before the first is used
#pragma unroll
  for (int i = 0; i < Q / GATE_WARPS; ++i) {
    const int j = warp + GATE_WARPS * i;
    v[i] = 0.f;
    if (j < sg.len && h < a.H) {
      const int64_t at = (int64_t)(sg.tok0 + j) * a.lddt + h;
      v[i] = a.dt_f32 ? static_cast<const float*>(a.dt)[at] : to_f(static_cast<const __nv_bfloat16*>(a.dt)[at]);
    }
  }
#pragma unroll
  for (int i = 0; i < Q / GATE_WARPS; ++i) {
    const int j = warp + GATE_WARPS * i;
    const float x = v[i] + bias;
    sdt[j][lane] = j >= sg.len ? 0.f : a.softplus ? softplus_f(x) : x;
  }
  __syncthreads();
#pragma unroll 1
  for (int k = warp; k < 32 && h0 + k < a.H; k += GATE_WARPS) {
    const float A = a.A[h0 + k] * LOG2E;
    float dt[4], ss[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dt[i] = sdt[4 * lane + i][k];
    float run = 0.f;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      ss[i] = run;
      run += gate_log2(dt[i], A);
    }
    float after = run;  // inclusive sums from the last lane down
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const float v = __shfl_down_sync(0xffffffffu, after, m);
      if (lane + m < 32) after += v;
    }
    after = __shfl_down_sync(0xffffffffu, after, 1);
    if (lane == 31) after = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) ss[i] += after;
    const float end = __shfl_sync(0xffffffffu, ss[3], lane | 7);
    float* to = gates + ((int64_t)blockIdx.x * a.H + h0 + k) * GATES + 4 * lane;
    *reinterpret_cast<float4*>(to) = make_float4(ss[0], ss[1], ss[2], ss[3]);
    *reinterpret_cast<float4*>(to + Q) = make_float4(dt[0], dt[1], dt[2], dt[3]);
    if (lane < 24)
      *reinterpret_cast<float4*>(to + 2 * Q) = make_float4(dt[0] * ex2(ss[0] - end), dt[1] * ex2(ss[1] - end),
                                                         dt[2] * ex2(ss[2] - end), dt[3] * ex2(ss[3] - end));
  }
}

// Pieces [c0, c0 + n) of row j of a tile block to zero.
template <int N>
__device__ __forceinline__ void clear_pieces(unsigned char* tile, int j, int c0) {
#pragma unroll
  for (int c = 0; c < N; ++c) *reinterpret_cast<uint4*>(tile + piece(j, c0 + c)) = make_uint4(0u, 0u, 0u, 0u);
}

// w_j times the pieces [c0, c0 + N) of token row j (in `x`), as three blocks `stride` bytes apart.
template <int N>
__device__ __forceinline__ void build_xw(const uint4 (&x)[N], unsigned char* xw, int stride, int j, int c0, float w) {
  const uint64_t ww = pack2(w, w);
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const uint32_t at = piece(j, c0 + c);
    uint4 h, m, l;
    split3(mul2(widen2(x[c].x), ww), h.x, m.x, l.x);
    split3(mul2(widen2(x[c].y), ww), h.y, m.y, l.y);
    split3(mul2(widen2(x[c].z), ww), h.z, m.z, l.z);
    split3(mul2(widen2(x[c].w), ww), h.w, m.w, l.w);
    *reinterpret_cast<uint4*>(xw + at) = h;
    *reinterpret_cast<uint4*>(xw + stride + at) = m;
    *reinterpret_cast<uint4*>(xw + 2 * stride + at) = l;
  }
}

// ---------------------------------------------------------------------------
// The walk: one block per (segment, head, 64 columns of the state).
//   warp 0: the MMAs of U and of Yo's first terms of S0;  warp 1: those of CB, Yd and
//   Yo's second terms
//   warp 2: TMA loads;  warp 3: TMA stores of the outputs
//   groups 0, 1 (four warps each): M from CB (16 of each 32 columns each)
//   groups 2, 3: the state (32 columns each)
//   groups 4, 5: w x and the outputs (32 columns each)
// Every role runs through the chunks on its own; barriers hand the buffers
// over.  An MMA of 64 columns with both operands in shared memory takes as long
// as one of 96 (it waits for A): the three operands of U sit side by side as one
// of 192 columns.
// S0's second terms take the place of the first once Yo has read those (there is no
// room for both), while U's products run.  Yo's second products come before Yd, whose M
// takes longer to form: after Yd 458 us for the prompt below, by warp 0 after U 447, so 439.
// Bound by shared memory's 128 bytes a clock, beside issue: a chunk moves about 480 KB
// through it (TMA writes 80, the MMAs' operands 285, the roles' own 115), 3750 of the
// 5200 clk it takes.  One prompt of 32768 tokens of 64 heads x 64 columns x 128 rows in 29
// chunks a segment: 320 us (278 with one BF16 number each of M and S0; as four roles of
// one warp each with every wait's failure path in line 582).
// ---------------------------------------------------------------------------
constexpr int WALK_THREADS = 28 * 32;
// TMEM columns: CB (16 of them a step of 16 K, over which M is written: the first
// terms of its pairs over 8, the second over the next 8), U (the three terms'
// products), Yo, Yd.
constexpr uint32_t T_CB = 0, T_U = 128, T_YO = 320, T_YD = 384;

struct WalkSmem {
  unsigned char B[2][2 * BLK], C[2][2 * BLK], X[2][BLK];
  unsigned char xw[3][BLK];  // w x in three terms
  unsigned char S[BLK];      // S0: the first, then, once Yo has read them, the second terms of its pairs
  float gates[2][GATES];
  // [2]: by the chunk's parity, where a role may wait a chunk apart from the others
  uint64_t bc_full[2], bc_empty[2], x_full[2], x_empty[2], xw_full[2], staged[2];
  uint64_t cb_full, m_full, u_full, u_empty, s_full, yo_full, y_full, y_empty, done[2];
  uint64_t s2_full, yo2_full;  // the second terms of S0
  uint32_t tmem;
  int abort;
  Seg seg;
};

__global__ void __launch_bounds__(WALK_THREADS, 1) k_ssm_walk(const __grid_constant__ TcArgs ta) {
  extern __shared__ __align__(1024) unsigned char ssm_smem[];  // tiles are swizzled in 1024-byte atoms
  WalkSmem& s = *reinterpret_cast<WalkSmem*>(ssm_smem);
  const SsmArgs& a = ta.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int per = a.H * ta.pblocks;
  const int hp = blockIdx.x % per, h = hp / ta.pblocks, p0 = (hp % ta.pblocks) * PT, sid = blockIdx.x / per;
  const int nblk = a.NS > 64 ? 2 : 1, ksteps = (a.NS + 15) / 16;
  if (warp == 0) {
    const Seg sg = find_segment(a.cu, a.N, ta.lseg, sid);
    if (lane == 0) {
      s.seg = sg;
      s.abort = 0;
      for (int i = 0; i < 2; ++i) {
        tc::mbar_init(&s.bc_full[i], 1);
        tc::mbar_init(&s.bc_empty[i], 2);
        tc::mbar_init(&s.x_full[i], 1);
        tc::mbar_init(&s.x_empty[i], 1 + 8 + 1);
        tc::mbar_init(&s.staged[i], 8);
        tc::mbar_init(&s.xw_full[i], 8);
        tc::mbar_init(&s.done[i], 1);
      }
      tc::mbar_init(&s.u_full, 1);
      tc::mbar_init(&s.u_empty, 8);
      tc::mbar_init(&s.s_full, 8);
      tc::mbar_init(&s.yo_full, 1);
      tc::mbar_init(&s.s2_full, 8);
      tc::mbar_init(&s.yo2_full, 1);
      tc::mbar_init(&s.y_full, 1);
      tc::mbar_init(&s.y_empty, 8);
      tc::mbar_init(&s.cb_full, 1);
      tc::mbar_init(&s.m_full, 8);
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
  const Seg sg = uniform(s.seg);
  const uint32_t tmem = __shfl_sync(0xffffffffu, s.tmem, 0);
  const int nch = (sg.len + Q - 1) / Q;
  volatile int* ab = &s.abort;
  const int quad = warp & 3, r = 32 * quad + lane;         // TMEM lanes of the warp; row of the thread
  const uint32_t trow = tmem + ((uint32_t)(32 * quad) << 16);
  const int group = (warp >> 2) - 1, half = group & 1;
  const float A = a.A[h] * LOG2E;
  // descriptor address units (16 bytes): a stage of B or C, a block, a step of
  // 16 K rows (MN-major); a step of 16 K elements (K-major: 32 bytes, four a block)
  constexpr uint32_t stage2 = 2 * BLK / 16, stage1 = BLK / 16, step = 2048 / 16;
  auto kmaj = [](int k) { return (uint32_t)((k >> 2) * (BLK / 16) + (k & 3) * 2); };

  if (warp == 0) {
    constexpr uint32_t i_yo = tc::idesc_bf16(128, PT) | tc::kIdescTransposeB;
    constexpr uint32_t i_u = tc::idesc_bf16(128, 3 * PT) | tc::kIdescTransposeB | kIdescTransposeA;
    const uint32_t d_c = desc_lo(s.C[0]), d_b = desc_lo(s.B[0]), d_w = desc_lo(s.xw[0]), d_s = desc_lo(s.S);
    bool ok = true;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
      const uint32_t b = c & 1;
      // Yo = C S0, the first terms
      ok = warp_wait(&s.s_full, c & 1, ab) && warp_wait(&s.bc_full[b], (c >> 1) & 1, ab);
      if (c > 0) ok = ok && warp_wait(&s.y_empty, (c - 1) & 1, ab);
      if (!ok) break;
      tc::tc_fence_after();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < ksteps) mma_ss(tmem + T_YO, d_c + b * stage2 + kmaj(k), d_s + k * step, i_yo, k > 0);
      commit(&s.yo_full);
      // U = B^T (w x)
      ok = warp_wait(&s.xw_full[b], (c >> 1) & 1, ab);
      if (c > 0) ok = ok && warp_wait(&s.u_empty, (c - 1) & 1, ab);
      if (!ok) break;
      tc::tc_fence_after();
#pragma unroll
      for (int k = 0; k < 8; ++k) mma_ss(tmem + T_U, d_b + b * stage2 + k * step, d_w + k * step, i_u, k > 0);
      commit(&s.u_full);
      commit(&s.bc_empty[b]);
    }
    // no MMA is in flight when the block ends
    if (nch > 0) {
      commit(&s.done[0]);
      tc::mbar_wait(&s.done[0], 0);
    }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t i_cb = tc::idesc_bf16(128, 128);
    constexpr uint32_t i_yd = tc::idesc_bf16(128, PT) | tc::kIdescTransposeB;
    constexpr uint32_t i_yo = tc::idesc_bf16(128, PT) | tc::kIdescTransposeB;
    const uint32_t d_c = desc_lo(s.C[0]), d_b = desc_lo(s.B[0]), d_x = desc_lo(s.X[0]), d_s = desc_lo(s.S);
    bool ok = true;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
      const uint32_t b = c & 1;
      // CB = C B^T, once Yd has read the M in its columns
      ok = warp_wait(&s.bc_full[b], (c >> 1) & 1, ab);
      if (c > 0) ok = ok && warp_wait(&s.y_full, (c - 1) & 1, ab);
      if (!ok) break;
      tc::tc_fence_after();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < ksteps) mma_ss(tmem + T_CB, d_c + b * stage2 + kmaj(k), d_b + b * stage2 + kmaj(k), i_cb, k > 0);
      commit(&s.cb_full);
      // Yo += C S0, the second terms (written once the first terms' products are there)
      if (!warp_wait(&s.s2_full, c & 1, ab)) break;
      tc::tc_fence_after();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < ksteps) mma_ss(tmem + T_YO, d_c + b * stage2 + kmaj(k), d_s + k * step, i_yo, true);
      commit(&s.yo2_full);
      commit(&s.bc_empty[b]);
      // Yd = M x (M waited for x; the rows past the end are cleared with w x)
      ok = warp_wait(&s.m_full, c & 1, ab);
      if (sg.len - c * Q < Q) ok = ok && warp_wait(&s.xw_full[b], (c >> 1) & 1, ab);
      if (c > 0) ok = ok && warp_wait(&s.y_empty, (c - 1) & 1, ab);
      if (!ok) break;
      tc::tc_fence_after();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        mma_ts(tmem + T_YD, tmem + T_CB + 16 * k, d_x + b * stage1 + k * step, i_yd, k > 0);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        mma_ts(tmem + T_YD, tmem + T_CB + 16 * k + 8, d_x + b * stage1 + k * step, i_yd, true);
      commit(&s.y_full);  // (Yo's products came before)
      commit(&s.x_empty[b]);
    }
    if (nch > 0) {
      commit(&s.done[1]);
      tc::mbar_wait(&s.done[1], 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    if (lane == 0) {
      const int grp = h / (a.H / a.G);
      int bc = 0, x = 0;  // chunks asked for
#pragma unroll 1
      for (int c = 0; c < nch; ++c) {
        const int b = c & 1, row = sg.tok0 + c * Q;
        if (c >= 2 && !wait_or_abort(&s.bc_empty[b], ((c >> 1) - 1) & 1, ab)) break;
        tc::mbar_arrive_expect_tx(&s.bc_full[b], (uint32_t)(2 * nblk * BLK));
#pragma unroll 1
        for (int k = 0; k < nblk; ++k) {
          tc::tma_load_3d(s.C[b] + k * BLK, &ta.c_map, 64 * k, grp, row, &s.bc_full[b]);
          tc::tma_load_3d(s.B[b] + k * BLK, &ta.b_map, 64 * k, grp, row, &s.bc_full[b]);
        }
        bc = c + 1;
        if (c >= 2 && !wait_or_abort(&s.x_empty[b], ((c >> 1) - 1) & 1, ab)) break;
        tc::mbar_arrive_expect_tx(&s.x_full[b], (uint32_t)(BLK + sizeof(s.gates[0])));
        tc::tma_load_3d(s.X[b], &ta.x_map, p0, h, row, &s.x_full[b]);
        if (c == 0) previous_ended();  // the gates come from the kernel before
        tc::bulk_load(s.gates[b], gates_of(ta, sg.chunk0 + c, h).p, sizeof(s.gates[0]), &s.x_full[b]);
        x = c + 1;
      }
      // no copy is in flight when the block ends
#pragma unroll 1
      for (int c = max(0, bc - 2); c < bc; ++c) tc::mbar_wait(&s.bc_full[c & 1], (c >> 1) & 1);
#pragma unroll 1
      for (int c = max(0, x - 2); c < x; ++c) tc::mbar_wait(&s.x_full[c & 1], (c >> 1) & 1);
    }
    __syncwarp();
  } else if (warp == 3) {
    bool ok = true;
#pragma unroll 1
    for (int c = 0; c < nch && ok; ++c) {
      const int b = c & 1;
      ok = warp_wait(&s.staged[b], (c >> 1) & 1, ab);
      if (ok && lane == 0) {
        if (sg.len - c * Q >= Q) {  // a whole chunk; a partial one was stored row by row
          asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n" ::"l"(
                           reinterpret_cast<uint64_t>(&ta.out_map)),
                       "r"(p0), "r"(h), "r"(sg.tok0 + c * Q), "r"(tc::smem_u32(s.X[b]))
                       : "memory");
          asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
          asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
        }
        arrive(&s.x_empty[b]);
      }
      __syncwarp();
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
    __syncwarp();
  } else if (group == 0 || group == 1) {
    // M: thread = row r; column blocks b < quad by factors 2^(ss[end of b] - ss_r)
    // colf_j, both at most 1; b == quad from the difference; zero above the diagonal
    const int j0 = 16 * half;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
      const int st = c & 1;
      const Gates g{s.gates[st]};
      if (!warp_wait(&s.x_full[st], (c >> 1) & 1, ab) || !warp_wait(&s.cb_full, c & 1, ab)) break;
      tc::tc_fence_after();
      const float sr = g.ss()[r];
      const uint32_t cb = trow + T_CB + j0;
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        uint32_t v[16], m[16];  // first terms, second terms
        if (b < quad) {
          tc::tmem_ld16(cb + 32 * b, v);
          const float rf = ex2(g.ss()[32 * b + 31] - sr);
          const uint64_t rr = pack2(rf, rf);
          ulonglong2 cf[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            cf[j] = *reinterpret_cast<const ulonglong2*>(g.colf() + 32 * b + j0 + 4 * j);
            cf[j].x = mul2(cf[j].x, rr);
            cf[j].y = mul2(cf[j].y, rr);
          }
          wait_ld(v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            split2(mul2(pair_of(v + 4 * j), cf[j].x), m[2 * j], m[8 + 2 * j]);
            split2(mul2(pair_of(v + 4 * j + 2), cf[j].y), m[2 * j + 1], m[8 + 2 * j + 1]);
          }
        } else if (b == quad) {
          tc::tmem_ld16(cb + 32 * b, v);
          float f[16];
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 sj = *reinterpret_cast<const float4*>(g.ss() + 32 * b + j0 + j);
            const float4 dj = *reinterpret_cast<const float4*>(g.dt() + 32 * b + j0 + j);
            f[j] = dj.x * ex2(sj.x - sr);
            f[j + 1] = dj.y * ex2(sj.y - sr);
            f[j + 2] = dj.z * ex2(sj.z - sr);
            f[j + 3] = dj.w * ex2(sj.w - sr);
          }
          wait_ld(v);
#pragma unroll
          for (int j = 0; j < 16; j += 2)
            split2(pack2(j0 + j <= lane ? __uint_as_float(v[j]) * f[j] : 0.f,
                         j0 + j + 1 <= lane ? __uint_as_float(v[j + 1]) * f[j + 1] : 0.f),
                   m[j / 2], m[8 + j / 2]);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) m[j] = 0u;
        }
        tc::tmem_st16(cb + 32 * b, m);  // over columns just read
      }
      tc::tmem_wait_st();
      tc::tc_fence_before();
      warp_arrive(&s.m_full);
    }
  } else if (group == 2 || group == 3) {
    // state row n = r, columns p0 + 32 half + [0, 32)
    const int pc = p0 + 32 * half;
    uint64_t S[16];
    const float* start = nullptr;
    previous_ended();  // a segment's start state, too
    // Of a split document every start state comes from k_ssm_merge, the first segment's too:
    // ht may be h0, and the block of the last segment writes it whenever it is done.
    if (sg.nseg > 1) start = ta.seg + (((int64_t)sg.slot * a.H + h) * a.NS + r) * a.P + pc;
    else if (a.h0) start = a.h0 + (((int64_t)sg.doc * a.H + h) * a.NS + r) * a.P + pc;
#pragma unroll
    for (int q = 0; q < 16; q += 2) {
      ulonglong2 v = make_ulonglong2(0, 0);
      if (start && r < a.NS && pc + 2 * q < a.P) v = *reinterpret_cast<const ulonglong2*>(start + 2 * q);
      S[q] = v.x;
      S[q + 1] = v.y;
    }
    float gam = 0.f;
    bool ok = true;
    auto advance = [&](int c) {  // S = gam S + U of chunk c
      ok = warp_wait(&s.u_full, c & 1, ab);
      if (!ok) return;
      tc::tc_fence_after();
      const uint64_t gg = pack2(gam, gam), one = pack2(1.f, 1.f);
#pragma unroll
      for (int p = 0; p < 32; p += 8) {
        uint32_t u[8], v[8], w[8];
        tmem_ld8(trow + T_U + 32 * half + p, u);
        tmem_ld8(trow + T_U + PT + 32 * half + p, v);
        tmem_ld8(trow + T_U + 2 * PT + 32 * half + p, w);
        wait_ld(u);
        wait_ld(v);
        wait_ld(w);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          S[p / 2 + q] = fma2(gg, S[p / 2 + q],
                              fma2(one, pair_of(u + 2 * q), fma2(one, pair_of(v + 2 * q), pair_of(w + 2 * q))));
      }
      tc::tc_fence_before();
      warp_arrive(&s.u_empty);
    };
#pragma unroll 1
    for (int c = 0; c <= nch; ++c) {
      if (c > 0) advance(c - 1);
      if (!ok || c == nch) break;
      uint4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        v[q] = make_uint4(round2(S[4 * q]), round2(S[4 * q + 1]), round2(S[4 * q + 2]), round2(S[4 * q + 3]));
      ok = warp_wait(&s.x_full[c & 1], (c >> 1) & 1, ab);
      // the previous chunk's Yo has read the operand
      if (c > 0) ok = ok && warp_wait(&s.yo2_full, (c - 1) & 1, ab);
      if (!ok) break;
      gam = ex2(Gates{s.gates[c & 1]}.total(A));
      warp_arrive(&s.x_empty[c & 1]);
#pragma unroll
      for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(s.S + piece(r, 4 * half + q)) = v[q];
      tc::fence_proxy_async();
      warp_arrive(&s.s_full);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        v[q] = make_uint4(rest2(S[4 * q]), rest2(S[4 * q + 1]), rest2(S[4 * q + 2]), rest2(S[4 * q + 3]));
      ok = warp_wait(&s.yo_full, c & 1, ab);
      if (!ok) break;
#pragma unroll
      for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(s.S + piece(r, 4 * half + q)) = v[q];
      tc::fence_proxy_async();
      warp_arrive(&s.s2_full);
    }
    if (ok && sg.idx == sg.nseg - 1 && a.ht && r < a.NS) {
      float* to = a.ht + (((int64_t)sg.doc * a.H + h) * a.NS + r) * a.P + pc;
#pragma unroll
      for (int q = 0; q < 16; q += 2)
        if (pc + 2 * q < a.P) *reinterpret_cast<ulonglong2*>(to + 2 * q) = make_ulonglong2(S[q], S[q + 1]);
    }
  } else {
    // w x and the outputs of token row r, columns p0 + 32 half + [0, 32); x and the
    // decay from the chunk's start stay in registers from the one to the other
    const int pc = p0 + 32 * half;
    const float D = a.D ? a.D[h] : 0.f;
    const uint64_t DD = pack2(D, D);
    bool ok = true;
    uint4 x[4];
    uint64_t ee = 0;
#pragma unroll 1
    for (int c = -1; c < nch; ++c) {
      if (c >= 0) {
        const int len = sg.len - c * Q;
        __nv_bfloat16* out = a.out + ((int64_t)(sg.tok0 + c * Q + r) * a.H + h) * a.P + pc;
        ok = warp_wait(&s.y_full, c & 1, ab);
        if (!ok) break;
        tc::tc_fence_after();
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          uint32_t yo[8], yd[8], y[4];
          tmem_ld8(trow + T_YO + 32 * half + 8 * p, yo);
          tmem_ld8(trow + T_YD + 32 * half + 8 * p, yd);
          const uint32_t xs[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
          wait_ld(yo);
          wait_ld(yd);
#pragma unroll
          for (int z = 0; z < 4; ++z)
            y[z] = round2(fma2(DD, widen2(xs[z]), fma2(ee, pair_of(yo + 2 * z), pair_of(yd + 2 * z))));
          // a whole chunk's outputs take the place of x and leave by TMA
          const uint4 yv = make_uint4(y[0], y[1], y[2], y[3]);
          if (len >= Q) *reinterpret_cast<uint4*>(s.X[c & 1] + piece(r, 4 * half + p)) = yv;
          else if (r < len && pc + 8 * p < a.P) *reinterpret_cast<uint4*>(out + 8 * p) = yv;
        }
        tc::tc_fence_before();
        warp_arrive(&s.y_empty);
        tc::fence_proxy_async();
        warp_arrive(&s.staged[c & 1]);
      }
      if (c + 1 < nch) {  // w x of the next chunk, once U has read this one's
        const int n = (c + 1) & 1, len = sg.len - (c + 1) * Q;
        const Gates g{s.gates[n]};
        ok = warp_wait(&s.x_full[n], ((c + 1) >> 1) & 1, ab);
        if (c >= 0) ok = ok && warp_wait(&s.u_full, c & 1, ab);
        if (len < Q) ok = ok && warp_wait(&s.bc_full[n], ((c + 1) >> 1) & 1, ab);
        if (!ok) break;
        if (r >= len) {
          clear_pieces<4>(s.X[n], r, 4 * half);
          if (half < nblk) clear_pieces<8>(s.B[n] + half * BLK, r, 0);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) x[p] = *reinterpret_cast<const uint4*>(s.X[n] + piece(r, 4 * half + p));
        const float ss = g.ss()[r], w = g.dt()[r] * ex2(ss), e = ex2(g.total(A) - ss);
        ee = pack2(e, e);
        build_xw<4>(x, s.xw[0], BLK, r, 4 * half, w);
        tc::fence_proxy_async();
        warp_arrive(&s.xw_full[n]);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && s.abort) atomicExch(ta.err, 10);
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Summary of a segment (split documents only): its end state from a zero start,
//   U = B^T (w x) with w_j = dt_j exp(sum of the gates after j in the segment),
// over its chunks, last chunk first, and its total decay.
// A block takes two neighbours (head, 64 columns) of a group, or one where a group's
// number of them is odd; two share the chunks of B.
//   warps 0, 2: TMA of x and B;  warp 1: MMA;  warps 4-19: w x, eight for the first / second neighbour
//   (for the even / odd chunks where there is one), four for each half of a chunk
// w x goes in three BF16 terms; the first two have an accumulator each, the third
// joins the second's.  Of two neighbours the same terms lie side by side, so that
// one MMA of 256 columns and one of 128 read a piece of B twice, not four times:
// shared memory's bandwidth bounds the kernel.
// The tensor cores' FP32 accumulation truncates, a bias that grows with the
// number of products: after kBatch chunks the warps add the sums up in registers,
// while the other of two accumulators takes over.
// The same prompt: 106 us, 141 with one neighbour a block (a group of one head of 64
// columns takes 143).  Bound by shared memory: 352 KB a pair of chunks, 2750 of 3280 clk.
// ---------------------------------------------------------------------------
constexpr int SUM_THREADS = 640, SUM_STAGES = 2, kBatch = 4, kAhead = 6;
struct SumSmem {
  unsigned char B[SUM_STAGES][2 * BLK], X[SUM_STAGES][2][BLK];
  unsigned char xw[6][BLK];  // [term][neighbour], or [chunk parity][term]
  uint64_t x_full[SUM_STAGES], x_empty[SUM_STAGES], b_full[SUM_STAGES], b_empty[SUM_STAGES];
  uint64_t xw_full[2][2], xw_empty[2][2], acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int abort;
  Seg seg;
};

__global__ void __launch_bounds__(SUM_THREADS, 1) k_ssm_sum(const __grid_constant__ TcArgs ta) {
  extern __shared__ __align__(1024) unsigned char ssm_smem[];
  SumSmem& s = *reinterpret_cast<SumSmem*>(ssm_smem);
  const SsmArgs& a = ta.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int two = ta.pairs, per = two ? a.H * ta.pblocks / 2 : a.H * ta.pblocks;
  const int item = (blockIdx.x % per) << two, sid = blockIdx.x / per;  // the first neighbour
  const int grp = item / ta.pblocks / (a.H / a.G);
  const int nblk = a.NS > 64 ? 2 : 1;
  if (warp == 0) {
    const Seg sg = find_segment(a.cu, a.N, ta.lseg, sid);
    if (lane == 0) {
      s.seg = sg;
      s.abort = 0;
      for (int i = 0; i < SUM_STAGES; ++i) {
        tc::mbar_init(&s.x_full[i], 1);
        tc::mbar_init(&s.x_empty[i], 8 << two);
        tc::mbar_init(&s.b_full[i], 1);
        tc::mbar_init(&s.b_empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        for (int n = 0; n < 2; ++n) {
          tc::mbar_init(&s.xw_full[i][n], 4 << two);
          tc::mbar_init(&s.xw_empty[i][n], 1);
        }
        tc::mbar_init(&s.acc_full[i], 1);
        tc::mbar_init(&s.acc_empty[i], 8 << two);
      }
      tc::mbar_init(&s.done, 1);
      tc::mbar_fence_init();
    }
  }
  __syncthreads();
  const Seg sg = uniform(s.seg);
  next_may_start();
  previous_ended();
  if (sg.idx == sg.nseg - 1) return;  // no segment starts from this one's end
  if (warp == 1) {
    tc::tmem_alloc(&s.tmem, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s.tmem, 0);
  const int nch = sg.len / Q;  // a segment that is not its document's last holds whole chunks
  volatile int* ab = &s.abort;

  if (warp == 0 || warp == 2) {
    if (lane == 0) {
      const bool is_x = warp == 0;
      uint64_t* full = is_x ? s.x_full : s.b_full;
      uint64_t* empty = is_x ? s.x_empty : s.b_empty;
      int issued = 0;
#pragma unroll 1
      for (int k = 0, b = 0, ph = 1; k < nch; ++k) {
        const int row = sg.tok0 + (nch - 1 - k) * Q;
        if (k >= SUM_STAGES && !wait_or_abort(&empty[b], ph, ab)) break;
        tc::mbar_arrive_expect_tx(&full[b], (uint32_t)((is_x ? 1 + two : nblk) * BLK));
        if (is_x) {
#pragma unroll 1
          for (int n = 0; n <= two; ++n) {
            const int x = (item + n) % ta.pblocks * PT, y = (item + n) / ta.pblocks;
            tc::tma_load_3d(s.X[b][n], &ta.x_map, x, y, row, &full[b]);
            if (k + kAhead < nch) tc::tma_prefetch_3d(&ta.x_map, x, y, row - kAhead * Q);
          }
        } else {
#pragma unroll 1
          for (int q = 0; q < nblk; ++q) tc::tma_load_3d(s.B[b] + q * BLK, &ta.b_map, 64 * q, grp, row, &full[b]);
        }
        issued = k + 1;
        if (++b == SUM_STAGES) {
          b = 0;
          ph ^= 1;
        }
      }
      // no copy is in flight when the block ends
#pragma unroll 1
      for (int k = max(0, issued - SUM_STAGES); k < issued; ++k)
        tc::mbar_wait(&full[k % SUM_STAGES], (k / SUM_STAGES) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t i_hi = tc::idesc_bf16(128, 2 * PT << two) | tc::kIdescTransposeB | kIdescTransposeA;
    const uint32_t i_lo = tc::idesc_bf16(128, PT << two) | tc::kIdescTransposeB | kIdescTransposeA;
    const uint32_t d_b = desc_lo(s.B[0]), d_w = desc_lo(s.xw[0]);
    constexpr uint32_t blk = BLK / 16, step = 2048 / 16;
    const uint32_t lo = (2 << two) * blk, mid = PT << two;  // third terms; second terms' accumulators
    uint32_t b = 0;
    bool ok = true;
#pragma unroll 1
    for (int k = 0; k < nch && ok; ++k) {
      const int batch = k / kBatch, first = k % kBatch == 0;
      const uint32_t m = two ? 0 : k & 1, acc = tmem + (batch & 1) * 256;
      const uint32_t bb = d_b + b * 2 * blk, ww = d_w + m * 3 * blk;
      ok = warp_wait(&s.b_full[b], (k / SUM_STAGES) & 1, ab);
      if (first && batch >= 2) ok = ok && warp_wait(&s.acc_empty[batch & 1], ((batch >> 1) - 1) & 1, ab);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        ok = ok && warp_wait(&s.xw_full[m][half], (two ? k : k >> 1) & 1, ab);
        if (!ok) break;
        tc::tc_fence_after();
#pragma unroll
        for (int q = 4 * half; q < 4 * half + 4; ++q) mma_ss(acc, bb + q * step, ww + q * step, i_hi, !first || q > 0);
#pragma unroll
        for (int q = 4 * half; q < 4 * half + 4; ++q) mma_ss(acc + mid, bb + q * step, ww + lo + q * step, i_lo, true);
        commit(&s.xw_empty[m][half]);
      }
      if (k % kBatch == kBatch - 1 || k == nch - 1) commit(&s.acc_full[batch & 1]);
      commit(&s.b_empty[b]);
      b = b == SUM_STAGES - 1 ? 0 : b + 1;
    }
    commit(&s.done);
    tc::mbar_wait(&s.done, 0);
    __syncwarp();
  } else if (warp >= 4) {
    // group g: half a chunk's rows, a row's 32 columns a thread; state row j's 32 columns
    const int g = (warp - 4) >> 2, half = g & 1, j = (tid - 128) & 127, r = 64 * half + (j & 63), c0 = 4 * (j >> 6);
    const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const int n = two ? g >> 1 : 0, h = (item + n) / ta.pblocks, p0 = (item + n) % ta.pblocks * PT;
    const bool sums = two || g < 2;
    const float A = a.A[h] * LOG2E;
    float tail = 0.f;  // the gates after this chunk
    uint64_t S[PT / 4];
#pragma unroll
    for (int q = 0; q < PT / 4; ++q) S[q] = 0;
    auto drain = [&](int batch) {
      if (!warp_wait(&s.acc_full[batch & 1], (batch >> 1) & 1, ab)) return false;
      tc::tc_fence_after();
#pragma unroll
      for (int p = 0; p < PT / 2; p += 8) {
        uint32_t u[8], v[8];
        tmem_ld8(trow + (batch & 1) * 256 + n * PT + PT / 2 * half + p, u);
        tmem_ld8(trow + (batch & 1) * 256 + (PT << two) + n * PT + PT / 2 * half + p, v);
        wait_ld(u);
        wait_ld(v);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          S[p / 2 + q] = add2(add2(pair_of(u + 2 * q), pair_of(v + 2 * q)), S[p / 2 + q]);
      }
      tc::tc_fence_before();
      warp_arrive(&s.acc_empty[batch & 1]);
      return true;
    };
    bool ok = true;
    int drained = 0;
    float dt, ss, total;  // a chunk ahead
    auto gates = [&](int k) {
      const Gates ga = gates_of(ta, sg.chunk0 + nch - 1 - k, h);
      dt = ga.dt()[r], ss = ga.ss()[r], total = ga.total(A);
    };
    gates(0);
#pragma unroll 1
    for (int k = 0, b = 0, ph = 0; k < nch; ++k) {
      const float w = dt * ex2(ss + tail);
      tail += total;
      gates(min(k + 1, nch - 1));
      if (two || (k & 1) == g >> 1) {
        const int m = two ? 0 : k & 1, use = two ? k : k >> 1;
        ok = warp_wait(&s.x_full[b], ph, ab);
        if (!ok) break;
        uint4 x[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = *reinterpret_cast<const uint4*>(s.X[b][n] + piece(r, c0 + c));
        warp_arrive(&s.x_empty[b]);
        ok = use < 1 || warp_wait(&s.xw_empty[m][half], (use - 1) & 1, ab);
        if (!ok) break;
        build_xw<4>(x, s.xw[3 * m + n], BLK << two, r, c0, w);
        tc::fence_proxy_async();
        warp_arrive(&s.xw_full[m][half]);
      }
      if (++b == SUM_STAGES) {
        b = 0;
        ph ^= 1;
      }
      // a batch behind: its last product has had time to finish
      if (sums && k % kBatch == kBatch - 1 && k >= 2 * kBatch - 1) {
        ok = drain(drained++);
        if (!ok) break;
      }
    }
    if (sums) {
#pragma unroll 1
      while (ok && drained * kBatch < nch) ok = drain(drained++);
      if (ok && j < a.NS) {
        float* to = ta.seg + (((int64_t)sg.slot * a.H + h) * a.NS + j) * a.P;
#pragma unroll
        for (int q = 0; q < PT / 4; q += 2) {
          const int p = p0 + PT / 2 * half + 2 * q;
          if (p < a.P) *reinterpret_cast<ulonglong2*>(to + p) = make_ulonglong2(S[q], S[q + 1]);
        }
      }
      if (j == 0 && half == 0 && p0 == 0) ta.gsum[(int64_t)sg.slot * a.H + h] = tail;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && s.abort) atomicExch(ta.err, 10);
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

// The start states of split documents' segments, in place of the segments' own
// end states: S[s + 1] = 2^gsum[s] S[s] + U[s].  One thread per state element.
__global__ void __launch_bounds__(256) k_ssm_merge(const __grid_constant__ TcArgs ta) {
  const SsmArgs& a = ta.a;
  const int64_t elems = (int64_t)a.NS * a.P;
  const int eblocks = (int)((elems + 1023) / 1024);
  const int e0 = (blockIdx.x % eblocks) * 1024 + threadIdx.x * 4, h = (blockIdx.x / eblocks) % a.H;
  const int d = blockIdx.x / eblocks / a.H;
  // the document's first segment: the segments of the split documents before it
  int before = 0;
  for (int i = threadIdx.x; i < d; i += 256) {
    const int ch = (a.cu[i + 1] - a.cu[i] + Q - 1) / Q;
    before += ch > ta.lseg ? (ch + ta.lseg - 1) / ta.lseg : 0;
  }
  __shared__ int sums[8];
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) before += __shfl_xor_sync(0xffffffffu, before, m);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = before;
  __syncthreads();
  before = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) before += sums[i];
  next_may_start();
  previous_ended();
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

// Whether the summaries' blocks take two neighbouring (head, 64 columns) of a group.
static int ssm_pairs(int H, int P, int G) { return H / G * ((P + 63) / 64) % 2 == 0; }

// Whole documents while they keep the SMs evenly busy; else the segment length
// with the least estimated time, in chunk steps of one walking block (2.5 us): kStart
// steps to start a block, kSum for a chunk of a summary (of one (head, 64 columns) or of
// two; 0.7 and 0.48 give the same plans' times).  One document of 32768 tokens of 64 heads:
// 442 us in 9 segments, 680 whole (64 blocks); 8192 tokens of 16 heads 57 us against 175;
// three documents of 65536 together of 16 heads 230 against 464.
SsmPlan ssm_tc_plan(int H, int P, int NS, int G, int N, const int32_t* cu) {
  const int pairs = ssm_pairs(H, P, G);
  const double kStart = 3.0, kSum = pairs ? 0.8 : 0.55;
  const int64_t items = (int64_t)H * ((P + 63) / 64);
  const double sms = 152.0;
  int64_t nc = 0, most = 0;
  int64_t gate_chunks = 0;
  for (int i = 0; i < N; ++i) {
    const int64_t ch = (cu[i + 1] - (int64_t)cu[i] + Q - 1) / Q;
    nc += ch;
    gate_chunks += std::max<int64_t>(ch, 1);
    most = std::max(most, ch);
  }
  SsmPlan best{(int)std::max<int64_t>(most, 1), N, 0, 0, false, 0};
  double cost = std::max((double)(nc + kStart * N) * items / sms, most + kStart);
  best.chunks = gate_chunks;
  best.scratch = up256((size_t)gate_chunks * H * GATES * sizeof(float));
  // (nothing to gain where whole documents come near to even work)
  if (cost < 1.1 * nc * items / sms) return best;
  // pieces of the longest document; only documents longer than the shortest piece are
  // looked at again, those of one length together
  const int64_t shortest = std::max<int64_t>(4, (most + 255) / 256);
  std::vector<std::pair<int64_t, int64_t>> longer;  // (chunks, documents that have as many), longest first
  try {
    std::vector<int64_t> chunks;
    for (int i = 0; i < N; ++i) {
      const int64_t ch = (cu[i + 1] - (int64_t)cu[i] + Q - 1) / Q;
      if (ch > shortest) chunks.push_back(ch);
    }
    std::sort(chunks.begin(), chunks.end(), std::greater<int64_t>());
    for (int64_t ch : chunks) {
      if (longer.empty() || longer.back().first != ch) longer.push_back({ch, 0});
      ++longer.back().second;
    }
  } catch (const std::bad_alloc&) {
    return best;  // (whole documents need no list)
  }
  int64_t last = 0;
  for (int64_t k = 2; k <= 256 && (most + k - 1) / k >= 4; ++k) {
    const int64_t L = (most + k - 1) / k;
    if (L == last) continue;
    last = L;
    int64_t ends = 0, split = 0;  // segments that another one follows, documents that have such
    for (const auto& d : longer) {
      if (d.first <= L) break;
      ends += ((d.first + L - 1) / L - 1) * d.second;
      split += d.second;
    }
    const int64_t nseg = N + ends;
    const double waves = (double)nseg * items / sms;
    const double walk = std::max((nc + kStart * nseg) * items / sms, (double)(L + kStart) * (int64_t)(waves + 0.999));
    const double sum = kSum * L * (int64_t)((double)(ends * items >> pairs) / sms + 0.999) + 2 * kStart;
    if (walk + sum < 0.95 * cost) {
      cost = walk + sum;
      best.lseg = (int)L;
      best.nseg = nseg;
      best.states = ends + split;
      best.split = true;
    }
  }
  if (best.split)
    best.scratch += up256((size_t)best.states * H * NS * P * sizeof(float)) + up256((size_t)best.states * H * sizeof(float));
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
        !token_map(&t.c_map, a.C, a.T, a.G, a.NS, a.T > 1 ? a.ldc : (uint64_t)a.G * a.NS * one) ||
        !token_map(&t.out_map, a.out, a.T, a.H, a.P, a.T > 1 ? (uint64_t)a.H * a.P : (uint64_t)a.H * a.P * one))
      return cudaErrorInvalidValue;
  }
  t.gates = static_cast<const float*>(scratch);
  {
    ProfScope ps("ssm_gates", st, (double)a.T * a.H);
    k_ssm_gates<<<dim3((unsigned)plan.chunks, (a.H + 31) / 32), GATE_WARPS * 32, 0, st>>>(a.cu, a, static_cast<float*>(scratch));
  }
  if (cudaError_t e = cudaGetLastError()) return e;
  char* rest = static_cast<char*>(scratch) + up256((size_t)plan.chunks * a.H * GATES * sizeof(float));
  const unsigned grid = (unsigned)(plan.nseg * a.H * t.pblocks);
  t.pairs = ssm_pairs(a.H, a.P, a.G);
  constexpr int sm_walk = (int)sizeof(WalkSmem), sm_sum = (int)sizeof(SumSmem);
  static_assert(sm_walk <= 232448 && sm_sum <= 232448, "227 KB of shared memory a block");
  if (plan.split) {
    t.seg = reinterpret_cast<float*>(rest);
    t.gsum = reinterpret_cast<float*>(rest + up256((size_t)plan.states * a.H * a.NS * a.P * sizeof(float)));
    cudaFuncSetAttribute(k_ssm_sum, cudaFuncAttributeMaxDynamicSharedMemorySize, sm_sum);
    {
      ProfScope ps("ssm_sum", st, (double)a.T * a.H);
      if (cudaError_t e = launch_early(k_ssm_sum, dim3(grid >> t.pairs), SUM_THREADS, sm_sum, st, t)) return e;
    }
    ProfScope ps("ssm_merge", st);
    const unsigned mb = (unsigned)(((int64_t)a.NS * a.P + 1023) / 1024) * a.H * a.N;
    if (cudaError_t e = launch_early(k_ssm_merge, dim3(mb), 256, 0, st, t)) return e;
  }
  cudaFuncSetAttribute(k_ssm_walk, cudaFuncAttributeMaxDynamicSharedMemorySize, sm_walk);
  ProfScope ps("ssm_walk", st, (double)a.T * a.H);
  return launch_early(k_ssm_walk, dim3(grid), WALK_THREADS, sm_walk, st, t);
}

}  // namespace gdr
