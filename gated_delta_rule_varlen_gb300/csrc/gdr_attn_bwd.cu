// gdr_attn_bwd.cu -- softmax attention's backward on the tensor cores (formulas:
// gdr_attn.cuh), in two kernels so that every sum has one owner and a fixed order:
//
//   k_attn_dq   a tile of 128 queries, its keys 128 at a time:
//               S = Q K^T, dP = dO V^T, dS = P (dP - delta) over S in tensor memory, dQ += dS K
//   k_attn_dkv  a tile of 128 keys of one key head, the queries of its heads 128 at a time:
//               S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
//
// Scores and probabilities are formed in both (seven products instead of five, but no sums
// across blocks).  P and dS are the A operands of their products, read from tensor memory in
// BF16 (2^-8 of each term at most, independently: where the keys share a large part, which
// cancels in dQ since a row of dS sums to zero, that part times the roundings stays);
// accumulators, P and dS before that are FP32.
//
// delta = dout . out of the rounded out is off by up to 2^-8 of |dout| |out|, which is nothing
// beside dS of probabilities spread over many keys, and all of it where one key has nearly all:
// dP - delta is small there.  What it is off by is sum dS, which comes with the tiles of dS: delta is
// put right for dK and dV, and a tile of dQ with a row that it matters to (put_right) is formed again by
// a second launch.  Of 8192 tokens of 16 heads of 128 the sums take 15 us of dQ, the second launch 19 for
// the few tiles that unit inputs leave it, and 298 for all of them (scores 4 times as large).  Where a tile of keys holds all that the queries see, delta is
// sum p dP from the start: with few keys |out| is like |v|.
//
// Bound by the products and their operands' way from shared memory: of 8192 tokens of 16
// heads over 4 of 128 columns dQ takes 298 us (three products, 1.4 PFLOP/s), dK and dV 354
// (four, 1.55 PFLOP/s; cuBLAS's measured rate is 1.9).  Measured and not kept: tiles three
// deep in dQ and two in dK and dV, so that elements and products of different tiles overlap
// (345 and 423 us: the elements' tensor memory traffic slows the products), the products of
// dK and dV from two warps (408), eight warps on the elements (323 and 417), every warp
// finding its items for itself (300 and 375).
//
// Rows past a document's end belong to another one: they are cleared where they are summed
// over (K for dQ, Q and dO for dK and dV).
#include "gdr_attn_tc.cuh"

namespace gdr {
namespace {

struct BwdArgs {
  CUtensorMap q_map, k_map, v_map, do_map;
  AttnArgs a;
  int pack;
  int parts;    // blocks that share a tile's sums
  float* part;  // their shares: dQ [parts][T][H][D], or dK and dV [2][parts][TK][HK][D]
  float4* sums; // of dQ's parts, [parts][H][T]: sum dS, sum P^2, half of sum dS^2, the delta that dS was formed with
  int items;    // dQ's tiles
  int* err;
};

// Sixteen warps on the elements of a tile, four on each quarter of its columns (of two
// warpgroups with halves each waited on its own loads and barriers), and one warpgroup of
// roles.
constexpr int QUARTERS = 4, WORKERS = 4 * QUARTERS, THREADS = 32 * WORKERS + 128;
constexpr int COLS = TILE / QUARTERS;

// One after another through a ring of tiles.
template <int ST>
struct Ring {
  int st = 0, ph = 0;
  __device__ __forceinline__ void step() {
    if (++st == ST) {
      st = 0;
      ph ^= 1;
    }
  }
};

// A tile of 128 rows to shared memory; the bytes are credited to bar (one lane).
template <int DB>
__device__ __forceinline__ void load_tile(unsigned char* to, const CUtensorMap* map, int head, int64_t token, uint64_t* bar) {
  tc::mbar_arrive_expect_tx(bar, DB * BLK);
#pragma unroll
  for (int c = 0; c < DB; ++c) tc::tma_load_3d(to + c * BLK, map, 64 * c, head, (int)token, bar);
}
// Rows [rows, 128) of a tile to zero (one warp).
template <int DB>
__device__ __forceinline__ void clear_rows(unsigned char* tile, int rows) {
  for (int e = rows * 8 + (threadIdx.x & 31); e < TILE * 8; e += 32)
#pragma unroll
    for (int c = 0; c < DB; ++c) *reinterpret_cast<uint4*>(tile + c * BLK + e * 16) = make_uint4(0, 0, 0, 0);
  tc::fence_proxy_async();
}
// A tile's products over the columns of two tiles in shared memory, ks steps of 16.
template <int DB>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id, int ks) {
#pragma unroll
  for (int k = 0; k < 4 * DB; ++k) {
    const uint32_t at = ((k >> 2) * BLK + (k & 3) * 32) >> 4;
    if (k < ks) mma_ss(d, a_lo + at, b_lo + at, id, k > 0);
  }
}
// Products over 128 rows of a tile in shared memory; A in tensor memory, BF16 pairs in the
// first half of each quarter's columns.
__device__ __forceinline__ void mma_sum(uint32_t d, uint32_t at, uint32_t b_lo, uint32_t id, bool more) {
#pragma unroll
  for (int k = 0; k < TILE / 16; ++k)
    mma_ts(d, at + (k >> 1) * COLS + (k & 1) * 8, b_lo + k * (16 * 128 >> 4), id, more || k > 0);
}
__device__ __forceinline__ uint32_t round_pair(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint64_t pair_at(const uint32_t* x) { return pack2(__uint_as_float(x[0]), __uint_as_float(x[1])); }
__device__ __forceinline__ void load_cols(uint32_t at, uint32_t (&x)[COLS]) {
  tc::tmem_ld32(at, x);
  tc::tmem_wait_ld();
  pin(x);
}
__device__ __forceinline__ void store_words(uint32_t at, const uint32_t (&x)[COLS]) {  // the first half of x
  uint32_t w[COLS / 2];
#pragma unroll
  for (int i = 0; i < COLS / 2; ++i) w[i] = x[i];
  tc::tmem_st16(at, w);
  tc::tmem_wait_st();
}
// 16 accumulator columns of a row, scaled, to 16 (or up to the row's end) elements, or, a
// share of them, to FP32.
__device__ __forceinline__ void store16(__nv_bfloat16* row, float* share, int c0, int D, uint32_t at, float f, bool any, bool live) {
  uint32_t o[16];
  if (any) {
    tc::tmem_ld16(at + c0, o);
    wait_ld(o);
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) o[k] = any ? __float_as_uint(__uint_as_float(o[k]) * f) : 0u;
  if (!live) return;
  if (share) {
#pragma unroll
    for (int k = 0; k < 16; k += 4)
      if (c0 + k < D) *reinterpret_cast<uint4*>(share + c0 + k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
    return;
  }
#pragma unroll
  for (int k = 0; k < 16; k += 8) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = round_pair(pair_at(o + k + 2 * e));
    if (c0 + k < D) *reinterpret_cast<uint4*>(row + c0 + k) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---------------------------------------------------------------------------
// dQ
// ---------------------------------------------------------------------------
// What a block works on at a time: a tile of queries, a part of its keys.
struct DqWork {
  AttnBlock b;
  int h0, hk, part, i1;
  TileRange all, r;
  __device__ __forceinline__ void find(const BwdArgs& ba, BlockFinder<true>& finder, int item) {
    const AttnArgs& a = ba.a;
    const int heads = 1 << ba.pack, tokens = TILE >> ba.pack, groups = a.H >> ba.pack;
    part = item % ba.parts;
    item /= ba.parts;
    b = finder.find(item / groups);
    h0 = item % groups * heads;
    hk = h0 / (a.H / a.HK);
    i1 = min(b.lq, b.first + tokens);
    all = tiles_of(a, b.lq, b.lk, b.first, i1);
    r = part_of(all, part, ba.parts);
  }
  __device__ __forceinline__ int steps() const { return max(0, r.hi - r.lo); }
};

template <int DB>
struct DqSmem {
  // a K tile is held from S until its dQ, a step later
  static constexpr int KS = DB == 2 ? 3 : 6, VS = DB == 2 ? 2 : 4;
  unsigned char Q[DB * BLK], dO[DB * BLK];
  unsigned char K[KS][DB * BLK], V[VS][DB * BLK];
  float part[QUARTERS][TILE];          // the quarters' shares of delta, or of what it is off by
  uint8_t squares_ds[TILE][QUARTERS];  // exponents
  WorkQueue<DqWork> queue;
  uint64_t q_full, do_full, q_empty, k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], cleared;
  uint64_t s_full[2], dp_full, dp_read, ds_full, dq_done[2], part_full, acc_full, acc_empty, done;
  uint32_t tmem;
  int abort;
};
constexpr int T_DP = 256, T_DQ = 384;  // (two tiles of S, and over them dS, before)

// The lowest bit of delta says that dQ has to be formed again with it.
__device__ __forceinline__ float marked(float delta, bool again) {
  return __uint_as_float((__float_as_uint(delta) & ~1u) | (again ? 1u : 0u));
}
__device__ __forceinline__ bool is_marked(float delta) { return (__float_as_uint(delta) & 1u) != 0; }
// delta put right by e = sum dS, which it was off by.  A row of dQ is then off by e |sum P k|: some |k| times
// the root of x = sum P^2 where the keys point in all directions, up to |k| where they share a part (which
// cancels in dQ, but not in this), so that an eighth of |k| is reckoned with at least.  The row is some |k|
// times the root of sum dS^2, of which y has half of the terms.  It is formed again where the first is more
// than 2^-9 of the second.  What stays is within 2^-9 of its terms' size, within 2^-6 where the keys are
// nearly one, and the root of two times that where the half's terms are the row (dS' own rounding: 2^-8 of
// each term).  Of unit inputs e is 2^-9 of the root in the mean: with a fourth of |k| reckoned with, one of 130
// rows was formed again; with an eighth, one of 40000.
__device__ __forceinline__ float put_right(float delta, float e, float x, float y) {
  return marked(delta + e, fabsf(e) * fmaxf(sqrtf(x), 0.125f) > sqrtf(2.f * y) * (1.f / 512.f) || y > 1e38f);
}
// What a block works on: one tile; one tile, for whose delta it goes through the keys once before;
// its own and those that it takes over; of every gridDim-th the marked ones, formed again.
enum Form { ONE_TILE, TWICE, TAKE_OVER, AGAIN };

template <int DB, int FORM>
__global__ void __launch_bounds__(THREADS, 1) k_attn_dq(const __grid_constant__ BwdArgs ba) {
  constexpr bool QUEUE = FORM == TAKE_OVER || FORM == AGAIN;  // several tiles, from the queue
  constexpr bool ROUGH = FORM == ONE_TILE || FORM == TAKE_OVER;  // delta of the rounded out, put right behind the keys
  using Smem = DqSmem<DB>;
  constexpr int KS = Smem::KS, VS = Smem::VS;
  extern __shared__ __align__(1024) unsigned char attn_smem[];
  Smem& s = *reinterpret_cast<Smem*>(attn_smem);
  const AttnArgs& a = ba.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* ab = &s.abort;
  if (warp == 1 && lane == 0)
    for (const CUtensorMap* map : {&ba.q_map, &ba.do_map, &ba.k_map, &ba.v_map}) prefetch_map(map);
  if (warp == 0) {
    if (lane == 0) {
      for (uint64_t* bar : {&s.q_full, &s.do_full, &s.cleared, &s.s_full[0], &s.s_full[1], &s.dp_full, &s.dq_done[0], &s.dq_done[1],
                            &s.acc_full})
        tc::mbar_init(bar, 1);
      for (uint64_t* bar : {&s.dp_read, &s.ds_full, &s.part_full, &s.acc_empty}) tc::mbar_init(bar, WORKERS);
      tc::mbar_init(&s.q_empty, 1 + WORKERS);
      tc::mbar_init(&s.done, 2);
      for (int i = 0; i < KS; ++i) {
        tc::mbar_init(&s.k_full[i], 1);
        tc::mbar_init(&s.k_empty[i], 1);
      }
      for (int i = 0; i < VS; ++i) {
        tc::mbar_init(&s.v_full[i], 1);
        tc::mbar_init(&s.v_empty[i], 1);
      }
      s.queue.init(3 + WORKERS);
      s.abort = 0;
      tc::mbar_fence_init();
    }
    __syncwarp();
    tc::tmem_alloc(&s.tmem, 512);
    tc::tmem_relinquish();
  }
  const int heads = 1 << ba.pack, tokens = TILE >> ba.pack;
  DqWork w;
  if constexpr (FORM != AGAIN) previous_ended();
  // All that came before this kernel has ended.  (Blocks of several tiles do not let the next kernel
  // in: its waits for delta would count their time.)
  if constexpr (!QUEUE) next_may_start();
  if constexpr (!QUEUE) {  // (one item, which every warp finds for itself)
    BlockFinder<true> finder(a, tokens);
    w.find(ba, finder, (int)blockIdx.x);
  }
  // Whether a row of the tile is marked (a warp).
  auto to_do = [&](const DqWork& t) {
    bool any = false;
    if (t.r.lo < t.r.hi)
      for (int row = lane; row < TILE; row += 32) {
        const int token = t.b.first + (row >> ba.pack);
        if (token < t.b.lq) any = any || is_marked(a.delta[(int64_t)(t.h0 + (row & (heads - 1))) * a.T + t.b.q0 + token]);
      }
    return __any_sync(0xffffffffu, any) != 0;
  };
  // Those of the block's first tiles, which its warps look at side by side (in the quarters' places).
  constexpr int KNOWN = FORM == AGAIN ? (int)sizeof(s.part) : 0;
  uint8_t* known = reinterpret_cast<uint8_t*>(s.part);
  if constexpr (FORM == AGAIN) {
    BlockFinder<true> finder(a, tokens);
    bool waited = false;
    for (int i = warp; i < KNOWN; i += THREADS / 32) {
      const int64_t item = blockIdx.x + (int64_t)i * gridDim.x;
      if (item >= ba.items) break;
      w.find(ba, finder, (int)item);
      if (!waited) previous_ended();  // (delta is there)
      waited = true;
      known[i] = to_do(w);
    }
    if (!waited) previous_ended();
  }
  int taken = 0;
  auto next_item = [&](bool ask) {
    if constexpr (QUEUE) return s.queue.take(taken, w, ab, ask);
    else return taken++ == 0;
  };
  auto steps = [&] { return (w.r.hi - w.r.lo) * (FORM == TWICE && w.r.hi - w.r.lo > 1 ? 2 : 1); };  // tiles of keys
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s.tmem;

  if (warp >= WORKERS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
    if (warp == WORKERS) {  // loads
      Ring<KS> kr;
      Ring<VS> vr;
      int g = 0, k = 0, cleared = 0;  // tiles, items so far
      bool ok = true;
      while (ok && next_item(true)) {
        const AttnBlock& b = w.b;
        if (w.r.lo >= w.r.hi) continue;
        if (k > 0 && !warp_wait(&s.q_empty, (k - 1) & 1, ab)) break;
        ++k;
        if (lane == 0) {
          load_tile<DB>(s.Q, &ba.q_map, w.h0, b.q0 + b.first, &s.q_full);
          load_tile<DB>(s.dO, &ba.do_map, w.h0, b.q0 + b.first, &s.do_full);
        }
        __syncwarp();
        for (int j = w.r.lo, left = steps(); left > 0; --left, j = j + 1 < w.r.hi ? j + 1 : w.r.lo, ++g) {
          const int rows = b.lk - j * TILE;
          const bool clear = rows < TILE;
          ok = g < KS || warp_wait(&s.k_empty[kr.st], kr.ph ^ 1, ab);
          if (!ok) break;
          if (lane == 0) load_tile<DB>(s.K[kr.st], &ba.k_map, w.hk, b.k0 + j * TILE, clear ? &s.cleared : &s.k_full[kr.st]);
          __syncwarp();
          if (clear) {
            ok = warp_wait(&s.cleared, cleared++ & 1, ab);
            if (!ok) break;
            clear_rows<DB>(s.K[kr.st], rows);
            warp_arrive(&s.k_full[kr.st]);
          }
          kr.step();
          ok = g < VS || warp_wait(&s.v_empty[vr.st], vr.ph ^ 1, ab);
          if (!ok) break;
          if (lane == 0) load_tile<DB>(s.V[vr.st], &ba.v_map, w.hk, b.k0 + j * TILE, &s.v_full[vr.st]);
          __syncwarp();
          vr.step();
        }
      }
      if (s.abort) {  // given up: the copies in flight land before the block ends
        for (int n = max(0, g + 1 - KS); n <= g; ++n) wait_some(&s.k_full[n % KS], (n / KS) & 1);
        for (int n = max(0, g - VS); n < g; ++n) wait_some(&s.v_full[n % VS], (n / VS) & 1);
        if (cleared > 0) wait_some(&s.cleared, (cleared - 1) & 1);
        if (k > 0) {
          wait_some(&s.q_full, (k - 1) & 1);
          wait_some(&s.do_full, (k - 1) & 1);
        }
      }
    } else if (warp == WORKERS + 1) {  // S and dP
      const uint32_t id_s = tc::idesc_bf16(TILE, TILE);
      const int ks = (a.D + 15) / 16;
      const uint32_t q_lo = desc_lo(s.Q), do_lo = desc_lo(s.dO);
      Ring<KS> kr;
      Ring<VS> vr;
      int g = 0, k = 0;
      bool ok = true;
      while (ok && next_item(false)) {
        if (w.r.lo >= w.r.hi) continue;
        ok = warp_wait_all(ab, Phase{&s.q_full, (uint32_t)k & 1}, Phase{&s.do_full, (uint32_t)k & 1});
        ++k;
        for (int left = steps(); left > 0 && ok; --left, ++g) {
          // S takes the place of dS two tiles ago, dP that of the last dP
          const Phase kp{&s.k_full[kr.st], (uint32_t)kr.ph}, vp{&s.v_full[vr.st], (uint32_t)vr.ph};
          ok = warp_wait_all(ab, kp, g >= 2 ? Phase{&s.dq_done[g & 1], (uint32_t)(g / 2 - 1) & 1} : kp);
          if (!ok) break;
          tc::tc_fence_after();  // (another warp issued the products that read dS)
          mma_rows<DB>(tmem + (g & 1) * TILE, q_lo, desc_lo(s.K[kr.st]), id_s, ks);
          commit(&s.s_full[g & 1]);
          kr.step();
          ok = warp_wait_all(ab, vp, g >= 1 ? Phase{&s.dp_read, (uint32_t)(g - 1) & 1} : vp);
          if (!ok) break;
          tc::tc_fence_after();
          mma_rows<DB>(tmem + T_DP, do_lo, desc_lo(s.V[vr.st]), id_s, ks);
          commit(&s.dp_full);
          commit(&s.v_empty[vr.st]);
          vr.step();
        }
        if (QUEUE) commit(&s.q_empty);
      }
      commit(&s.done);
      wait_some(&s.done, 0);
    } else if (warp == WORKERS + 2) {  // dQ: its waits cost the others nothing
      const int ks = (a.D + 15) / 16;
      const uint32_t id_d = tc::idesc_bf16(TILE, 16 * ks) | tc::kIdescTransposeB;
      Ring<KS> kr;
      int g = 0, k = 0;
      bool ok = true;
      while (ok && next_item(false)) {
        if (w.r.lo >= w.r.hi) continue;
        if (QUEUE && k > 0) ok = warp_wait(&s.acc_empty, (k - 1) & 1, ab);
        ++k;
        for (int left = steps(); left > 0 && ok; --left, ++g) {
          ok = warp_wait(&s.ds_full, g & 1, ab);
          if (!ok) break;
          tc::tc_fence_after();
          const int n = w.r.hi - w.r.lo;  // (of the steps for delta alone only the barriers go on)
          if (left <= n) mma_sum(tmem + T_DQ, tmem + (g & 1) * TILE, desc_lo(s.K[kr.st]), id_d, left < n);
          commit(&s.dq_done[g & 1]);
          commit(&s.k_empty[kr.st]);
          kr.step();
        }
        commit(&s.acc_full);
      }
      commit(&s.done);
      wait_some(&s.done, 0);
    } else {
      if constexpr (QUEUE) {
        BlockFinder<true> finder(a, tokens);
        auto make = [&](int item) {
          w.find(ba, finder, item);
          return w;
        };
        if constexpr (FORM == AGAIN)
          s.queue.run_those(ab, ba.items, make, known, KNOWN, to_do);
        else
          s.queue.run(ab, make);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;\n");  // (512 x 104 + 128 x 64 = 640 x 96; with 96 the sums spill)
    // a row a thread, of S and dP a quarter's columns
    const int quarter = warp >> 2, row = tid & 127, c0 = COLS * quarter;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const float c = a.scale * LOG2E;
    const uint64_t cc = pack2(c, c);
    auto squares_p = reinterpret_cast<uint8_t(*)[QUARTERS]>(s.part[0]);  // (the first quarter's own sum stays in registers)
    bool ok = true;
    int g = 0, k = 0;
    while (ok && next_item(false)) {
      const AttnBlock& b = w.b;
      const bool one = w.all.hi - w.all.lo == 1, any = w.r.lo < w.r.hi;  // one: the queries' keys fit one tile
      const int token = b.first + (row >> ba.pack), h = w.h0 + (row & (heads - 1));
      const int64_t at = b.q0 + token;
      const bool live = token < b.lq;
      const float lse = live ? a.lse_in[h * a.T + at] : -INFINITY;
      const float base = lse == -INFINITY ? -INFINITY : -lse * LOG2E;  // (rows that see nothing: p = 0)
      const uint64_t bb = pack2(base, base);
      const KeyRange kr = keys_of(a, token, b.lq, b.lk);
      const KeyRange seen{keys_of(a, w.i1 - 1, b.lq, b.lk).lo, keys_of(a, b.first, b.lq, b.lk).hi};  // keys every row sees
      float delta = FORM == AGAIN && live ? a.delta[h * a.T + at] : 0.f;
      auto exchange = [&](float mine) {  // delta of all quarters
        s.part[quarter][row] = mine;
        warp_arrive(&s.part_full);
        ok = ok && warp_wait(&s.part_full, 0, ab);  // (two exchanges a tile of queries)
        delta = (s.part[0][row] + s.part[1][row]) + (s.part[2][row] + s.part[3][row]);
      };
      // delta = sum p dP / sum p of all quarters, through the tensor memory that dQ comes to later.
      auto settle = [&](uint64_t pd, uint64_t ps) {
        uint32_t x[16] = {__float_as_uint(sum_of(pd)), __float_as_uint(sum_of(ps))};
        tc::tmem_st16(lanes + T_DQ + 16 * quarter, x);
        tc::tmem_wait_st();
        tc::tc_fence_before();
        warp_arrive(&s.part_full);
        ok = ok && warp_wait(&s.part_full, 0, ab);
        tc::tc_fence_after();
        float d = 0.f, all = 0.f;
#pragma unroll
        for (int i = 0; i < QUARTERS; ++i) {
          uint32_t y[8];
          tmem_ld8(lanes + T_DQ + 16 * i, y);
          wait_ld(y);
          d += __uint_as_float(y[0]);
          all += __uint_as_float(y[1]);
        }
        delta = all == 0.f ? 0.f : d / all;
      };
      if (any) {
        constexpr int PIECES = DB * 8 / QUARTERS;  // of 8 elements of a row
        uint4 o[PIECES];
        const bool given = !ROUGH || one;  // no delta of out
        const __nv_bfloat16* out = a.o + (at * a.H + h) * a.D;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          const int d = (quarter * PIECES + i) * 8;
          o[i] = !given && live && d < a.D ? *reinterpret_cast<const uint4*>(out + d) : make_uint4(0, 0, 0, 0);
        }
        // this tile's dO (the last one's place is free); nobody reads the last one's sums any more
        const Phase there{&s.do_full, (uint32_t)k & 1};
        ok = warp_wait_all(ab, there, QUEUE && k > 0 ? Phase{&s.acc_empty, (uint32_t)(k - 1) & 1} : there);
        if (!given) {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < PIECES; ++i) {
            const int pc = quarter * PIECES + i;
            const uint4 v = *reinterpret_cast<const uint4*>(s.dO + (pc >> 3) * BLK + piece(row, pc & 7));
            const uint32_t x[4] = {o[i].x, o[i].y, o[i].z, o[i].w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) sum = fmaf(bf_lo(x[e]), bf_lo(y[e]), fmaf(bf_hi(x[e]), bf_hi(y[e]), sum));
          }
          exchange(sum);
        }
        if (QUEUE) warp_arrive(&s.q_empty);
      }
      uint64_t off = 0;          // sum dS: what delta is off by
      uint64_t pp = 0, dd = 0;   // sum P^2, of every other pair sum dS^2
      uint64_t pd = 0, ps = 0;   // sum P dP, sum P
#pragma unroll 1
      for (int j = w.r.lo, left = steps(); left > 0; --left, j = j + 1 < w.r.hi ? j + 1 : w.r.lo, ++g) {
        const bool ahead = FORM == TWICE && left > w.r.hi - w.r.lo;  // for delta alone
        const uint32_t ts = lanes + (g & 1) * TILE + c0;
        ok = ok && warp_wait(&s.s_full[g & 1], (g >> 1) & 1, ab);
        if (!ok) break;
        tc::tc_fence_after();
        uint64_t p[COLS / 2];
        {
          uint32_t x[COLS];
          load_cols(ts, x);
#pragma unroll
          for (int i = 0; i < COLS / 2; ++i) {
            float e, f;
            unpack2(fma2(pair_at(x + 2 * i), cc, bb), e, f);
            p[i] = pack2(ex2(e), ex2(f));
          }
          if (j * TILE < seen.lo || (j + 1) * TILE > seen.hi) {
            const int lo = kr.lo - j * TILE - c0, hi = kr.hi - j * TILE - c0;
#pragma unroll
            for (int i = 0; i < COLS / 2; ++i) {
              float e, f;
              unpack2(p[i], e, f);
              p[i] = pack2(2 * i >= lo && 2 * i < hi ? e : 0.f, 2 * i + 1 >= lo && 2 * i + 1 < hi ? f : 0.f);
            }
          }
          if constexpr (ROUGH) {
#pragma unroll
            for (int i = 0; i < COLS / 2; ++i) pp = fma2(p[i], p[i], pp);
          }
        }
        ok = warp_wait(&s.dp_full, g & 1, ab);
        if (!ok) break;
        tc::tc_fence_after();
        uint32_t x[COLS];
        load_cols(lanes + T_DP + c0, x);
        tc::tc_fence_before();
        warp_arrive(&s.dp_read);
        if (b.lk - j * TILE < TILE) {  // keys past the document's end: whatever V holds there
#pragma unroll
          for (int i = 0; i < COLS; ++i)
            if (c0 + i >= b.lk - j * TILE) x[i] = 0u;
        }
        if (FORM == TWICE && (one || ahead)) {
#pragma unroll
          for (int i = 0; i < COLS / 2; ++i) {
            pd = fma2(p[i], pair_at(x + 2 * i), pd);
            ps = add2(ps, p[i]);
          }
          if (one || left - 1 == w.r.hi - w.r.lo) settle(pd, ps);
          if (!ok) break;
          if (ahead) {
            tc::tc_fence_before();
            warp_arrive(&s.ds_full);
            continue;
          }
        } else if (ROUGH && one) {
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < COLS / 2; ++i) sum[i & 1] = fma2(p[i], pair_at(x + 2 * i), sum[i & 1]);
          exchange(sum_of(add2(sum[0], sum[1])));
          if (!ok) break;
        }
        const uint64_t minus = pack2(-delta, -delta);
#pragma unroll
        for (int i = 0; i < COLS / 2; ++i) {
          const uint64_t ds = mul2(p[i], add2(pair_at(x + 2 * i), minus));
          if constexpr (ROUGH) {
            off = add2(off, ds);
            if (i % 2 == 0) dd = fma2(ds, ds, dd);  // (of all pairs: 312 us instead of 298)
          }
          x[i] = round_pair(ds);
        }
        store_words(ts, x);
        tc::tc_fence_before();
        warp_arrive(&s.ds_full);
      }
      if (!ok) break;
      if (any) {
        ok = warp_wait(&s.acc_full, k & 1, ab);
        if (!ok) break;
        tc::tc_fence_after();
        ++k;
      }
      // The other quarters' sums reach the first: sum dS in their places, of the sums of squares the
      // exponents, a byte each.  (All dS of the tile were there, and delta's shares read, for acc_full.)
      const float my_off = sum_of(off), my_pp = sum_of(pp), my_dd = sum_of(dd);
      if (ROUGH && any) {
        if (quarter > 0) {
          s.part[quarter][row] = my_off;
          squares_p[row][quarter] = (uint8_t)(__float_as_uint(my_pp) >> 23);
          s.squares_ds[row][quarter] = (uint8_t)(__float_as_uint(my_dd) >> 23);
        }
        warp_arrive(&s.part_full);
      }
      const int64_t to = (at * a.H + h) * a.D;
      float* share = ba.parts > 1 ? ba.part + w.part * a.T * a.H * a.D + to : nullptr;
#pragma unroll
      for (int i = 0; i < DB; ++i) store16(a.dq + to, share, DB * 16 * quarter + 16 * i, a.D, lanes + T_DQ, a.scale, any, live);
      if (ROUGH && any) {
        if (quarter == 0) {
          ok = warp_wait(&s.part_full, 1, ab);
          if (!ok) break;
          float e = my_off, x = my_pp, y = my_dd;
#pragma unroll
          for (int i = 1; i < QUARTERS; ++i) {
            e += s.part[i][row];
            x += __uint_as_float((uint32_t)squares_p[row][i] << 23 | 0x400000u);
            y += __uint_as_float((uint32_t)s.squares_ds[row][i] << 23);
          }
          if (live) {
            if (ba.parts > 1) ba.sums[(w.part * a.H + h) * a.T + at] = make_float4(e, x, y, delta);
            else a.delta[h * a.T + at] = put_right(delta, e, x, y);
          }
        }
      } else if (FORM == TWICE && any) {
        if (live && quarter == 0) a.delta[h * a.T + at] = delta;
      } else if (FORM != AGAIN && live && quarter == 0) {  // no keys, or none of this part
        if (ba.parts > 1) ba.sums[(w.part * a.H + h) * a.T + at] = make_float4(0.f, 0.f, 0.f, 0.f);
        else a.delta[h * a.T + at] = 0.f;
      }
      if (QUEUE && any) {
        tc::tc_fence_before();
        warp_arrive(&s.acc_empty);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && s.abort) atomicExch(ba.err, 11);
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// delta of a query whose keys are in parts, from the parts' sums.
__global__ void __launch_bounds__(256) k_attn_delta(const float4* __restrict__ sums, int parts, int64_t n, float* delta) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  previous_ended();
  if (i >= n) return;
  float e = 0.f, x = 0.f, y = 0.f, d = 0.f;
  for (int p = 0; p < parts; ++p) {
    const float4 s = sums[p * n + i];
    e += s.x;
    x += s.y;
    y += s.z;
    if (s.w != 0.f) d = s.w;  // (the same of all parts that have keys; zero of the others)
  }
  delta[i] = put_right(d, e, x, y);
}

// ---------------------------------------------------------------------------
// dK, dV
// ---------------------------------------------------------------------------
// What a block works on at a time: a tile of keys, a part of the tiles of queries (of all its
// heads, `per` tiles each from t0 on) that see them.
struct DkvWork {
  AttnBlock b;
  int hk, part, off, last, t0, per, n, g0, first;
  __device__ __forceinline__ void find(const BwdArgs& ba, BlockFinder<false>& finder, int item) {
    const AttnArgs& a = ba.a;
    const int G = a.H / a.HK;
    part = item % ba.parts;
    item /= ba.parts;
    b = finder.find(item / a.HK);
    hk = item % a.HK;
    off = b.lk - b.lq;
    last = min(b.lk, b.first + TILE) - 1;
    const TileRange r = query_tiles_of(a, b.lq, b.lk, b.first, last, TILE >> ba.pack);
    t0 = r.lo;
    per = r.hi - r.lo;
    const TileRange mine = part_of(TileRange{0, per * (G >> ba.pack)}, part, ba.parts);
    n = mine.hi - mine.lo;
    g0 = per ? mine.lo / per : 0;
    first = per ? mine.lo % per : 0;
  }
  __device__ __forceinline__ int steps() const { return n; }
};

template <int DB>
struct DkvSmem {
  // a Q tile is held until its dK, behind its dV
  static constexpr int QS = DB == 2 ? 3 : 6, OS = DB == 2 ? 2 : 4;
  unsigned char K[DB * BLK], V[DB * BLK];
  unsigned char Q[QS][DB * BLK], dO[OS][DB * BLK];
  alignas(16) float lse[2][TILE], delta[2][TILE];  // -lse log2 e, -delta
  WorkQueue<DkvWork> queue;
  uint64_t kv_full, kv_empty, q_full[QS], q_empty[QS], o_full[OS], o_empty[OS], q_cleared, o_cleared;
  uint64_t s_full, p_full, dp_full, ds_full, row_full[2], row_empty[2], acc_full, acc_empty, done;
  uint32_t tmem;
  int abort;
};
constexpr int T_DPT = 128, T_DK = 256, T_DV = 384;  // (S^T, and over it P^T, before)

template <int DB, bool QUEUE>
__global__ void __launch_bounds__(THREADS, 1) k_attn_dkv(const __grid_constant__ BwdArgs ba) {
  using Smem = DkvSmem<DB>;
  constexpr int QS = Smem::QS, OS = Smem::OS;
  extern __shared__ __align__(1024) unsigned char attn_smem[];
  Smem& s = *reinterpret_cast<Smem*>(attn_smem);
  const AttnArgs& a = ba.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* ab = &s.abort;
  if (warp == 1 && lane == 0)
    for (const CUtensorMap* map : {&ba.q_map, &ba.do_map, &ba.k_map, &ba.v_map}) prefetch_map(map);
  if (warp == 0) {
    if (lane == 0) {
      for (uint64_t* bar : {&s.kv_full, &s.kv_empty, &s.q_cleared, &s.o_cleared, &s.s_full, &s.dp_full, &s.row_full[0], &s.row_full[1],
                            &s.acc_full, &s.done})
        tc::mbar_init(bar, 1);
      for (uint64_t* bar : {&s.p_full, &s.ds_full, &s.row_empty[0], &s.row_empty[1], &s.acc_empty}) tc::mbar_init(bar, WORKERS);
      for (int i = 0; i < QS; ++i) {
        tc::mbar_init(&s.q_full[i], 1);
        tc::mbar_init(&s.q_empty[i], 1);
      }
      for (int i = 0; i < OS; ++i) {
        tc::mbar_init(&s.o_full[i], 1);
        tc::mbar_init(&s.o_empty[i], 1);
      }
      s.queue.init(3 + WORKERS);
      s.abort = 0;
      tc::mbar_fence_init();
    }
    __syncwarp();
    tc::tmem_alloc(&s.tmem, 512);
    tc::tmem_relinquish();
  }
  const int heads = 1 << ba.pack, tokens = TILE >> ba.pack, G = a.H / a.HK;
  DkvWork w;
  if constexpr (!QUEUE) {  // (one item, which every warp finds for itself)
    BlockFinder<false> finder(a, TILE);
    w.find(ba, finder, (int)blockIdx.x);
  }
  int taken = 0;
  auto next_item = [&](bool ask) {
    if constexpr (QUEUE) return s.queue.take(taken, w, ab, ask);
    else return taken++ == 0;
  };
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s.tmem;

  if (warp >= WORKERS) {
    if (warp == WORKERS) {  // loads
      Ring<QS> qr;
      Ring<OS> orr;
      int g = 0, k = 0, cleared = 0;  // tiles, items so far
      bool ok = true;
      while (ok && next_item(true)) {
        const AttnBlock& b = w.b;
        if (w.n == 0) continue;
        if (k > 0 && !warp_wait(&s.kv_empty, (k - 1) & 1, ab)) break;
        ++k;
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(&s.kv_full, 2 * DB * BLK);
          for (int c = 0; c < DB; ++c) {
            tc::tma_load_3d(s.K + c * BLK, &ba.k_map, 64 * c, w.hk, b.k0 + b.first, &s.kv_full);
            tc::tma_load_3d(s.V + c * BLK, &ba.v_map, 64 * c, w.hk, b.k0 + b.first, &s.kv_full);
          }
        }
        __syncwarp();
        for (int n = 0, hg = w.g0, t = w.first; n < w.n; ++n, ++g) {
          const int token = (w.t0 + t) * tokens, rows = (int)min((int64_t)TILE, (int64_t)(b.lq - token) << ba.pack);
          const bool clear = rows < TILE;
          const int h = w.hk * G + hg * heads;
          ok = g < QS || warp_wait(&s.q_empty[qr.st], qr.ph ^ 1, ab);
          if (!ok) break;
          if (lane == 0) load_tile<DB>(s.Q[qr.st], &ba.q_map, h, b.q0 + token, clear ? &s.q_cleared : &s.q_full[qr.st]);
          __syncwarp();
          if (clear) {
            ok = warp_wait(&s.q_cleared, cleared & 1, ab);
            if (!ok) break;
            clear_rows<DB>(s.Q[qr.st], rows);
            warp_arrive(&s.q_full[qr.st]);
          }
          ok = g < OS || warp_wait(&s.o_empty[orr.st], orr.ph ^ 1, ab);
          if (!ok) break;
          if (lane == 0) load_tile<DB>(s.dO[orr.st], &ba.do_map, h, b.q0 + token, clear ? &s.o_cleared : &s.o_full[orr.st]);
          __syncwarp();
          if (clear) {
            ok = warp_wait(&s.o_cleared, cleared & 1, ab);
            if (!ok) break;
            clear_rows<DB>(s.dO[orr.st], rows);
            warp_arrive(&s.o_full[orr.st]);
            ++cleared;
          }
          qr.step();
          orr.step();
          if (++t == w.per) {
            t = 0;
            ++hg;
          }
        }
      }
      if (s.abort) {  // given up: the copies in flight land before the block ends
        for (int n = max(0, g + 1 - QS); n <= g; ++n) wait_some(&s.q_full[n % QS], (n / QS) & 1);
        for (int n = max(0, g + 1 - OS); n <= g; ++n) wait_some(&s.o_full[n % OS], (n / OS) & 1);
        wait_some(&s.q_cleared, cleared & 1);
        wait_some(&s.o_cleared, cleared & 1);
        if (k > 0) wait_some(&s.kv_full, (k - 1) & 1);
      }
    } else if (warp == WORKERS + 1) {  // products
      const uint32_t id_s = tc::idesc_bf16(TILE, TILE);
      const int ks = (a.D + 15) / 16;
      const uint32_t id_d = tc::idesc_bf16(TILE, 16 * ks) | tc::kIdescTransposeB;
      const uint32_t k_lo = desc_lo(s.K), v_lo = desc_lo(s.V);
      Ring<QS> qr;
      Ring<OS> orr;
      int g = 0, k = 0, qst = 0, q2 = 0, ost = 0;
      bool ok = true;
      auto score = [&](int& at) {  // S^T of the next tile
        at = qr.st;
        mma_rows<DB>(tmem, k_lo, desc_lo(s.Q[at]), id_s, ks);
        commit(&s.s_full);
        qr.step();
      };
      auto grad = [&] {  // dP^T of the next tile
        ost = orr.st;
        mma_rows<DB>(tmem + T_DPT, v_lo, desc_lo(s.dO[ost]), id_s, ks);
        commit(&s.dp_full);
        orr.step();
      };
      while (ok && next_item(false)) {
        if (w.n == 0) continue;
        ok = warp_wait_all(ab, Phase{&s.kv_full, (uint32_t)k & 1}, Phase{&s.q_full[qr.st], (uint32_t)qr.ph});
        if (!ok) break;
        score(qst);
        ok = warp_wait(&s.o_full[orr.st], orr.ph, ab);
        if (!ok) break;
        grad();
        for (int n = 0; n < w.n && ok; ++n, ++g) {
          const bool more = n + 1 < w.n;
          const Phase pp{&s.p_full, (uint32_t)g & 1}, qp{&s.q_full[qr.st], (uint32_t)qr.ph};
          // (the last item's sums have been read before this one's begin)
          ok = QUEUE && n == 0 && k > 0 ? warp_wait_all(ab, pp, Phase{&s.acc_empty, (uint32_t)(k - 1) & 1}, more ? qp : pp)
                               : warp_wait_all(ab, pp, more ? qp : pp);
          if (!ok) break;
          tc::tc_fence_after();
          mma_sum(tmem + T_DV, tmem, desc_lo(s.dO[ost]), id_d, n > 0);
          commit(&s.o_empty[ost]);
          if (more) score(q2);
          const Phase dp{&s.ds_full, (uint32_t)g & 1};
          ok = warp_wait_all(ab, dp, more ? Phase{&s.o_full[orr.st], (uint32_t)orr.ph} : dp);
          if (!ok) break;
          tc::tc_fence_after();
          mma_sum(tmem + T_DK, tmem + T_DPT, desc_lo(s.Q[qst]), id_d, n > 0);
          commit(&s.q_empty[qst]);
          if (more) grad();
          else commit(&s.acc_full);
          if (QUEUE && (n + 2 == w.n || w.n == 1)) commit(&s.kv_empty);  // (S and dP of the last tile are on their way)
          qst = q2;
        }
        ++k;
      }
      commit(&s.done);
      wait_some(&s.done, 0);
    } else if (warp == WORKERS + 2) {  // lse and delta of a tile's queries
      previous_ended();  // (delta comes from k_attn_dq, beside whose last blocks this kernel begins)
      int g = 0;
      bool ok = true;
      while (ok && next_item(false)) {
        const AttnBlock& b = w.b;
        for (int n = 0, hg = w.g0, t = w.first; n < w.n; ++n, ++g) {
          float l[4], d[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = 4 * lane + e, token = (w.t0 + t) * tokens + (row >> ba.pack);
            const int64_t at = (int64_t)(w.hk * G + hg * heads + (row & (heads - 1))) * a.T + b.q0 + token;
            const bool live = token < b.lq;
            const float x = live ? a.lse_in[at] : -INFINITY;
            l[e] = x == -INFINITY ? x : -x * LOG2E;  // (queries that see nothing: p = 0)
            d[e] = live ? -a.delta[at] : 0.f;
          }
          ok = g < 2 || warp_wait(&s.row_empty[g & 1], ((g >> 1) - 1) & 1, ab);
          if (!ok) break;
          *reinterpret_cast<float4*>(&s.lse[g & 1][4 * lane]) = make_float4(l[0], l[1], l[2], l[3]);
          *reinterpret_cast<float4*>(&s.delta[g & 1][4 * lane]) = make_float4(d[0], d[1], d[2], d[3]);
          warp_arrive(&s.row_full[g & 1]);
          if (++t == w.per) {
            t = 0;
            ++hg;
          }
        }
      }
    } else {
      if constexpr (QUEUE) {
        BlockFinder<false> finder(a, TILE);
        s.queue.run(ab, [&](int item) {
          w.find(ba, finder, item);
          return w;
        });
      }
    }
  } else {
    // a key a thread, of S^T and dP^T a quarter's queries
    const int quarter = warp >> 2, row = tid & 127, c0 = COLS * quarter;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const float c = a.scale * LOG2E;
    const uint64_t cc = pack2(c, c);
    bool ok = true;
    int g = 0, k = 0;
    while (ok && next_item(false)) {
      const AttnBlock& b = w.b;
      const int key = b.first + row;
#pragma unroll 1
      for (int n = 0, t = w.first; n < w.n; ++n, ++g) {
        ok = warp_wait_all(ab, Phase{&s.row_full[g & 1], (uint32_t)(g >> 1) & 1}, Phase{&s.s_full, (uint32_t)g & 1});
        if (!ok) break;
        tc::tc_fence_after();
        uint64_t p[COLS / 2];
        uint32_t x[COLS];
        load_cols(lanes + c0, x);
        const ulonglong2* ls = reinterpret_cast<const ulonglong2*>(&s.lse[g & 1][c0]);
#pragma unroll
        for (int i = 0; i < COLS / 2; i += 2) {
          const ulonglong2 l = ls[i / 2];
          float e, f;
          unpack2(fma2(pair_at(x + 2 * i), cc, l.x), e, f);
          p[i] = pack2(ex2(e), ex2(f));
          unpack2(fma2(pair_at(x + 2 * i + 2), cc, l.y), e, f);
          p[i + 1] = pack2(ex2(e), ex2(f));
        }
        const int q0 = (w.t0 + t) * tokens;
        if (a.causal && (q0 + w.off < w.last || (a.window && (int64_t)q0 + tokens > (int64_t)b.first - w.off + a.window))) {
          // the queries of this tile that see the key: [lo, hi)
          const int64_t first = (int64_t)key - w.off - q0;
          const int lo = (int)min(max(first, (int64_t)0), (int64_t)tokens) << ba.pack;
          const int hi = a.window ? (int)min(max(first + a.window, (int64_t)0), (int64_t)tokens) << ba.pack : TILE;
#pragma unroll
          for (int i = 0; i < COLS / 2; ++i) {
            float e, f;
            unpack2(p[i], e, f);
            p[i] = pack2(c0 + 2 * i >= lo && c0 + 2 * i < hi ? e : 0.f, c0 + 2 * i + 1 >= lo && c0 + 2 * i + 1 < hi ? f : 0.f);
          }
        }
#pragma unroll
        for (int i = 0; i < COLS / 2; ++i) x[i] = round_pair(p[i]);
        store_words(lanes + c0, x);
        tc::tc_fence_before();
        warp_arrive(&s.p_full);
        ok = warp_wait(&s.dp_full, g & 1, ab);
        if (!ok) break;
        tc::tc_fence_after();
        load_cols(lanes + T_DPT + c0, x);
        const ulonglong2* ds = reinterpret_cast<const ulonglong2*>(&s.delta[g & 1][c0]);
#pragma unroll
        for (int i = 0; i < COLS / 2; i += 2) {
          const ulonglong2 d = ds[i / 2];
          x[i] = round_pair(mul2(p[i], add2(pair_at(x + 2 * i), d.x)));
          x[i + 1] = round_pair(mul2(p[i + 1], add2(pair_at(x + 2 * i + 2), d.y)));
        }
        store_words(lanes + T_DPT + c0, x);
        tc::tc_fence_before();
        warp_arrive(&s.ds_full);
        warp_arrive(&s.row_empty[g & 1]);
        if (++t == w.per) t = 0;
      }
      if (!ok) break;
      const bool any = w.n > 0;
      if (any) {
        ok = warp_wait(&s.acc_full, k++ & 1, ab);
        if (!ok) break;
        tc::tc_fence_after();
      }
      previous_ended();  // (nothing is written before; where there are queries delta has waited for it already)
      const int64_t to = ((int64_t)(b.k0 + key) * a.HK + w.hk) * a.D, all = a.TK * a.HK * a.D;
      float *dk = nullptr, *dv = nullptr;
      if (ba.parts > 1) {
        dk = ba.part + w.part * all + to;
        dv = dk + ba.parts * all;
      }
#pragma unroll
      for (int i = 0; i < DB; ++i) {
        store16(a.dk + to, dk, DB * 16 * quarter + 16 * i, a.D, lanes + T_DK, a.scale, any, key < b.lk);
        store16(a.dv + to, dv, DB * 16 * quarter + 16 * i, a.D, lanes + T_DV, 1.f, any, key < b.lk);
      }
      if (QUEUE && any) {
        tc::tc_fence_before();
        warp_arrive(&s.acc_empty);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && s.abort) atomicExch(ba.err, 11);
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// The shares of a sum, [parts][n], added in their order (blockIdx.y: dK, dV).
__global__ void __launch_bounds__(256) k_attn_sum(const float* __restrict__ part, int parts, int64_t n, __nv_bfloat16* x, __nv_bfloat16* y) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  previous_ended();
  if (i >= n) return;
  part += blockIdx.y * parts * n + i;
  float s[8] = {};
  for (int p = 0; p < parts; ++p, part += n) {
    const float4 u = *reinterpret_cast<const float4*>(part), v = *reinterpret_cast<const float4*>(part + 4);
    s[0] += u.x, s[1] += u.y, s[2] += u.z, s[3] += u.w, s[4] += v.x, s[5] += v.y, s[6] += v.z, s[7] += v.w;
  }
  vstore<__nv_bfloat16, 8>((blockIdx.y ? y : x) + i, s);
}

// early: begins beside the last blocks of the kernel before.
template <typename K>
cudaError_t go(K kernel, size_t smem, int64_t blocks, const BwdArgs& f, cudaStream_t st, bool early) {
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) return e;
  if (early) return launch_early(kernel, dim3((unsigned)blocks), THREADS, smem, st, f);
  kernel<<<dim3((unsigned)blocks), THREADS, smem, st>>>(f);
  return cudaGetLastError();
}
template <typename S>
constexpr size_t bytes_of() {
  static_assert(sizeof(S) <= 232448, "227 KB of shared memory a block");
  return sizeof(S);
}

}  // namespace

cudaError_t launch_attn_bwd(const AttnArgs& a, const AttnPlan& p, const int32_t* cu, const int32_t* cuk, float* scratch,
                            cudaStream_t st) {
  BwdArgs f{};
  f.a = a;
  f.err = device_error_ptr();
  if (!f.err) return cudaErrorUnknown;
  f.pack = p.pack;
  f.part = scratch;
  const int tokens = TILE >> f.pack;
  int64_t qblocks = 0, kblocks = 0;
  for (int i = 0; i < a.N; ++i) {
    qblocks += (cu[i + 1] - cu[i] + tokens - 1) / tokens;
    kblocks += (cuk[i + 1] - cuk[i] + TILE - 1) / TILE;
  }
  if (a.T > 0 && (!attn_map(&f.q_map, a.q, a.T, a.H, a.D, 1 << f.pack, tokens) ||
                  !attn_map(&f.do_map, a.dout, a.T, a.H, a.D, 1 << f.pack, tokens)))
    return cudaErrorInvalidValue;
  if (a.TK > 0 && (!attn_map(&f.k_map, a.k, a.TK, a.HK, a.D, 1, TILE) || !attn_map(&f.v_map, a.v, a.TK, a.HK, a.D, 1, TILE)))
    return cudaErrorInvalidValue;
  if (std::max(qblocks * (a.H >> f.pack) * p.dq, kblocks * a.HK * p.dkv) > sm_count()) attn_order(f.a, cuk);
  auto sum = [&](int64_t n, __nv_bfloat16* x, __nv_bfloat16* y) {  // (n is a multiple of 8, as D is)
    const int64_t blocks = (n / 8 + 255) / 256;
    if (f.parts == 1) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    ProfScope ps("attn_sum", st, (double)n / a.D);
    return launch_early(k_attn_sum, dim3((unsigned)blocks, y ? 2 : 1), 256, 0, st, f.part, f.parts, n, x, y);
  };
  // Blocks that take over others' items where there are enough of them: 16384 tokens of 16 heads
  // of 64, windows of 128 / 1024 / 4096: dQ 85 / 162 / 372 us against 114 / 185 / 390, dK and dV 77 /
  // 185 / 495 against 119 / 224 / 528; dK and dV of 8192 tokens of 16 heads of 128 over 4 key heads
  // (512 blocks) 352 against 340.
  if (qblocks > 0) {
    f.parts = p.dq;
    f.sums = reinterpret_cast<float4*>(scratch + p.dq * a.T * a.H * a.D);
    const int64_t blocks = qblocks * (a.H >> f.pack) * f.parts;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    f.items = (int)blocks;
    constexpr size_t b1 = bytes_of<DqSmem<1>>(), b2 = bytes_of<DqSmem<2>>();
    bool twice = false;
    int longest = 0;  // tiles of keys
    {
      ProfScope ps("attn_dq", st, (double)a.T * a.H);
      const int64_t sms = sm_count();
      auto pick = [&](auto form) {
        return a.D <= 64 ? go(k_attn_dq<1, decltype(form)::value>, b1, blocks, f, st, true)
                         : go(k_attn_dq<2, decltype(form)::value>, b2, blocks, f, st, true);
      };
      using std::integral_constant;
      // Where every block has one tile of few keys, going through them twice is quicker than the second
      // launch that the rounded out asks for: 4 heads of 64 / 128, documents of 300, 200, 157, 100 and 200
      // tokens 20 / 24 us against 28 / 32, one of 640 tokens (5 tiles of keys) 23.0 / 29.1 against 24.5 /
      // 30.5, of 900 (8 tiles) 32.7 / 40.5 against 31.5 / 38.7.
      if (blocks <= sms && f.parts == 1) {
        for (int i = 0; i < a.N; ++i)
          for (int lq = cu[i + 1] - cu[i], lk = cuk[i + 1] - cuk[i], at = 0; at < lq; at += tokens) {
            const TileRange r = tiles_of(a, lq, lk, at, std::min(lq, at + tokens));
            longest = std::max(longest, r.hi - r.lo);
          }
        twice = longest <= 6;
      }
      if (cudaError_t e = twice            ? pick(integral_constant<int, TWICE>{})
                          : blocks <= sms ? pick(integral_constant<int, ONE_TILE>{})
                                          : pick(integral_constant<int, TAKE_OVER>{}))
        return e;
    }
    if (f.parts > 1) {
      ProfScope ps("attn_delta", st, (double)a.T * a.H);
      const int64_t n = a.T * a.H, grid = (n + 255) / 256;
      if (grid > INT32_MAX) return cudaErrorInvalidValue;
      if (cudaError_t e = launch_early(k_attn_delta, dim3((unsigned)grid), 256, 0, st, f.sums, f.parts, n, a.delta)) return e;
    }
    if (!twice) {
      ProfScope ps("attn_dq_again", st);
      const int64_t grid = std::min<int64_t>(blocks, sm_count());
      if (cudaError_t e = a.D <= 64 ? go(k_attn_dq<1, AGAIN>, b1, grid, f, st, true) : go(k_attn_dq<2, AGAIN>, b2, grid, f, st, true)) return e;
    }
    if (cudaError_t e = sum(a.T * a.H * a.D, a.dq, nullptr)) return e;
  }
  if (kblocks > 0) {
    f.parts = p.dkv;
    const int64_t blocks = kblocks * a.HK * f.parts;
    {
      ProfScope ps("attn_dkv", st, (double)a.TK * a.HK);
      const bool queue = blocks > 4 * sm_count();
      constexpr size_t b1 = bytes_of<DkvSmem<1>>(), b2 = bytes_of<DkvSmem<2>>();
      // What it reads before it waits (the documents, q, k, v, dout) is there because dQ's kernel began
      // after all that came before; without queries there is no such kernel.
      const bool early = qblocks > 0;
      if (cudaError_t e = a.D <= 64 ? queue ? go(k_attn_dkv<1, true>, b1, blocks, f, st, early) : go(k_attn_dkv<1, false>, b1, blocks, f, st, early)
                          : queue   ? go(k_attn_dkv<2, true>, b2, blocks, f, st, early)
                                    : go(k_attn_dkv<2, false>, b2, blocks, f, st, early))
        return e;
    }
    if (cudaError_t e = sum(a.TK * a.HK * a.D, a.dk, a.dv)) return e;
  }
  return cudaSuccess;
}

}  // namespace gdr
