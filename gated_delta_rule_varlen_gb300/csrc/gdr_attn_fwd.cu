// gdr_attn_fwd.cu -- softmax attention's forward on the tensor cores (formulas:
// gdr_attn.cuh).
//
// A block has two tiles of 128 query rows of one key head and goes through its keys 128 at a
// time: S = Q K^T from shared memory into tensor memory, the softmax of a tile on one
// warpgroup, a row a thread (no exchange between threads), P in BF16 back over S, out += P V
// with P read from tensor memory.  While one tile's products run, the other tile's
// exponentials do.
//
// The running maximum is raised only when a tile's exceeds it by more than 8 (in powers of
// two): until then probabilities are up to 2^8 times what they are in the end, which FP32
// sums and BF16's exponent hold as well, and out needs no rescaling.  Sums of probabilities
// are of the unrounded ones in FP32.  P is rounded to BF16 (v's type, which the product
// needs): 2^-8 of each term at most, independently.
//
// Bound by the products' operand reads from shared memory (S takes both operands from there,
// 128 bytes a clock) and by what its one issuing warp waits: a step of a block's two tiles
// takes some 2700 clocks, its products 2048; one prompt of 32768 tokens of 16 heads over 4
// of 128 columns 2.9 ms, 1540 TFLOP/s (81% of cuBLAS's measured rate).  The exponentials
// cost nothing beside that (without them the same time).  Measured and not kept: products
// from a warp a tile (3.2 ms: the two streams of products slow each other), P handed over
// in halves (3.15).
//
// Rows of V past a document's keys are cleared, since they hold another document's values (a
// NaN there would pass through a zero probability).
#include "gdr_attn_tc.cuh"

namespace gdr {
namespace {

struct FwdArgs {
  CUtensorMap q_map, k_map, v_map;
  AttnArgs a;
  int pack;   // log2 of the heads side by side in a tile: row r is token r >> pack, head r & (2^pack - 1)
  int parts;  // blocks that share the keys of two tiles
  float *part_out, *part_lse;  // [parts][T][H][D], [parts][H][T]
  int* err;
};

constexpr int THREADS = 384;
// Tensor memory: S (and over it P) of the tiles, out of the tiles.
constexpr int T_S = 0, T_O = 256;

// What a block works on at a time: two tiles of queries of one head (or of several side by
// side), and a part of the keys that they see.
struct FwdWork {
  AttnBlock b;
  int h0, hk, part;
  TileRange r[2], all;
  bool dual;
  int step;
  __device__ __forceinline__ void find(const FwdArgs& fa, BlockFinder<true>& finder, int item) {
    const AttnArgs& a = fa.a;
    const int heads = 1 << fa.pack, tokens = TILE >> fa.pack, groups = a.H >> fa.pack;
    part = item % fa.parts;
    item /= fa.parts;
    b = finder.find(item / groups);
    h0 = item % groups * heads;
    hk = h0 / (a.H / a.HK);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int i0 = b.first + t * tokens;
      r[t] = tiles_of(a, b.lq, b.lk, i0, min(b.lq, i0 + tokens));
    }
    all = {min(r[0].lo, r[1].lo), max(r[0].hi, r[1].hi)};
    if (r[0].lo >= r[0].hi) all = r[1];
    if (r[1].lo >= r[1].hi) all = r[0];
    all = part_of(all, part, fa.parts);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      r[t].lo = max(r[t].lo, all.lo);
      r[t].hi = min(r[t].hi, all.hi);
    }
    // Where the second tile has no queries (few, of long keys), it takes every other key tile
    // of the first's: what waits on one pair of products goes on with the other.
    dual = b.first + tokens >= b.lq && r[0].hi - r[0].lo > 1;
    if (dual) r[1] = r[0];
    step = dual ? 2 : 1;
  }
  __device__ __forceinline__ int steps() const { return max(0, all.hi - all.lo); }
  __device__ __forceinline__ bool any(int t) const { return r[t].lo < r[t].hi; }
  __device__ __forceinline__ bool works(int t, int j) const {
    return dual ? ((j - all.lo) & 1) == t : j >= r[t].lo && j < r[t].hi;
  }
};

template <int DB>  // blocks of 64 columns
struct FwdSmem {
  static constexpr int STAGES = DB == 2 ? 5 : 10;
  unsigned char Q[2][DB * BLK];
  unsigned char KV[STAGES][DB * BLK];  // K and V tiles in turn
  uint64_t q_full[2], q_empty, full[STAGES], empty[STAGES], cleared;
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2], merged, swapped, done;
  WorkQueue<FwdWork> queue;
  float m[TILE], l[TILE];
  uint32_t tmem;
  int abort;
};

template <int DB, bool QUEUE>
__global__ void __launch_bounds__(THREADS, 1) k_attn_fwd(const __grid_constant__ FwdArgs fa) {
  using Smem = FwdSmem<DB>;
  constexpr int ST = Smem::STAGES;
  extern __shared__ __align__(1024) unsigned char attn_smem[];
  Smem& s = *reinterpret_cast<Smem*>(attn_smem);
  const AttnArgs& a = fa.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* ab = &s.abort;
  if (warp == 1 && lane == 0)
    for (const CUtensorMap* map : {&fa.q_map, &fa.k_map, &fa.v_map}) prefetch_map(map);
  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        tc::mbar_init(&s.q_full[i], 1);
        tc::mbar_init(&s.s_full[i], 1);
        tc::mbar_init(&s.p_full[i], 4);
        tc::mbar_init(&s.o_full[i], 1);
        tc::mbar_init(&s.o_empty[i], 4);
      }
      for (int i = 0; i < ST; ++i) {
        tc::mbar_init(&s.full[i], 1);
        tc::mbar_init(&s.empty[i], 1);
      }
      tc::mbar_init(&s.q_empty, 1);
      tc::mbar_init(&s.swapped, 4);
      tc::mbar_init(&s.cleared, 1);
      tc::mbar_init(&s.merged, 4);
      tc::mbar_init(&s.done, 1);
      s.queue.init(2 + 8);  // (loads, products, softmax)
      s.abort = 0;
      tc::mbar_fence_init();
    }
    __syncwarp();
    tc::tmem_alloc(&s.tmem, 512);
    tc::tmem_relinquish();
  }
  const int heads = 1 << fa.pack, tokens = TILE >> fa.pack;  // of a tile
  previous_ended();
  if constexpr (!QUEUE) next_may_start();
  FwdWork w;
  if constexpr (!QUEUE) {  // (one item, which every warp finds for itself)
    BlockFinder<true> finder(a, 2 * tokens);
    w.find(fa, finder, (int)blockIdx.x);
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

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
    if (warp == 8) {  // loads
      int i = 0, st = 0, ph = 0, cleared = 0, works = 0, duals = 0, q_loads[2] = {0, 0};
      bool ok = true;
      while (ok && next_item(true)) {
        const AttnBlock& b = w.b;
        if (w.all.lo >= w.all.hi) continue;
        if (works > 0) ok = warp_wait(&s.q_empty, (works - 1) & 1, ab);
        if (ok && duals > 0) ok = warp_wait(&s.swapped, (duals - 1) & 1, ab);
        if (!ok) break;
        ++works;
        duals += w.dual;
        for (int t = 0; t < 3 - w.step; ++t)
          if (w.any(t)) {
            ++q_loads[t];
            if (lane == 0) {
              tc::mbar_arrive_expect_tx(&s.q_full[t], DB * BLK);
              for (int c = 0; c < DB; ++c)
                tc::tma_load_3d(s.Q[t] + c * BLK, &fa.q_map, 64 * c, w.h0, b.q0 + b.first + t * tokens, &s.q_full[t]);
            }
          }
        __syncwarp();
        // K of the first `step` tiles, then V of each and K of the one `step` behind it
        auto load = [&](int j, bool isv) {
          if (i >= ST && !warp_wait(&s.empty[st], ph ^ 1, ab)) return false;
          const int rows = b.lk - j * TILE;
          uint64_t* bar = isv && rows < TILE ? &s.cleared : &s.full[st];
          if (lane == 0) {
            tc::mbar_arrive_expect_tx(bar, DB * BLK);
            for (int c = 0; c < DB; ++c)
              tc::tma_load_3d(s.KV[st] + c * BLK, isv ? &fa.v_map : &fa.k_map, 64 * c, w.hk, b.k0 + j * TILE, bar);
          }
          __syncwarp();
          ++i;
          if (isv && rows < TILE) {  // the document's last tile: clear what lies behind it
            if (!warp_wait(&s.cleared, cleared++ & 1, ab)) return false;
            for (int e = rows * 8 + lane; e < TILE * 8; e += 32)
              for (int c = 0; c < DB; ++c) *reinterpret_cast<uint4*>(s.KV[st] + c * BLK + e * 16) = make_uint4(0, 0, 0, 0);
            tc::fence_proxy_async();
            warp_arrive(&s.full[st]);
          }
          if (++st == ST) {
            st = 0;
            ph ^= 1;
          }
          return true;
        };
        for (int j = w.all.lo; j < w.all.lo + w.step && ok; ++j) ok = load(j, false);
        for (int j = w.all.lo; j < w.all.hi && ok; ++j) {
          ok = load(j, true);
          if (ok && j + w.step < w.all.hi) ok = load(j + w.step, false);
        }
      }
      if (!ok) {  // given up: the copies in flight land before the block ends
        for (int k = max(0, i - ST); k < i; ++k) wait_some(&s.full[k % ST], (k / ST) & 1);
        if (cleared > 0) wait_some(&s.cleared, (cleared - 1) & 1);
        for (int t = 0; t < 2; ++t)
          if (q_loads[t] > 0) wait_some(&s.q_full[t], (q_loads[t] - 1) & 1);
      }
    } else if (warp == 9) {  // products
      const uint32_t id_s = tc::idesc_bf16(TILE, TILE);
      const uint32_t id_o = tc::idesc_bf16(TILE, (a.D + 15) / 16 * 16) | tc::kIdescTransposeB;
      const int ks = (a.D + 15) / 16;
      bool ok = true;
      int used[2] = {0, 0}, outs[2] = {0, 0}, q_loads[2] = {0, 0};  // tiles, items, loads of Q so far
      int st = 0, ph = 0;  // the next tile of the ring
      auto next = [&] {
        const Phase p{&s.full[st], (uint32_t)ph};
        if (++st == ST) {
          st = 0;
          ph ^= 1;
        }
        return p;
      };
      auto stage = [&](const Phase& p) { return (int)(p.bar - s.full); };
      while (ok && next_item(false)) {
        const int j0 = w.all.lo, j1 = w.all.hi;
        if (j0 >= j1) continue;
        const uint32_t q_lo[2] = {desc_lo(s.Q[0]), desc_lo(s.Q[w.dual ? 0 : 1])};
        auto score = [&](int t, int at) {
          const uint32_t k_lo = desc_lo(s.KV[at]);
#pragma unroll
          for (int k = 0; k < 4 * DB; ++k) {
            const uint32_t o = ((k >> 2) * BLK + (k & 3) * 32) >> 4;
            if (k < ks) mma_ss(tmem + T_S + t * TILE, q_lo[t] + o, k_lo + o, id_s, k > 0);
          }
          commit(&s.s_full[t]);
        };
        Phase kp{};
        for (int t = 0; t < 3 - w.step && ok; ++t)
          if (w.any(t)) ok = warp_wait(&s.q_full[t], q_loads[t]++ & 1, ab);
        for (int j = j0; j < j0 + w.step && ok; ++j) {
          kp = next();
          ok = warp_wait(kp.bar, kp.parity, ab);
          if (!ok) break;
          for (int t = 0; t < 2; ++t)
            if (w.works(t, j)) score(t, stage(kp));
          commit(&s.empty[stage(kp)]);
          if (QUEUE && j == j1 - 1) commit(&s.q_empty);
        }
        bool first[2] = {true, true};
        for (int j = j0; j < j1 && ok; ++j) {
          const bool more = j + w.step < j1;
          const Phase vp = next();
          if (more) kp = next();
          bool loaded = false;  // V of this step, K of the next
          for (int t = 0; t < 2 && ok; ++t) {
            const bool here = w.works(t, j);
            const Phase pp{here ? &s.p_full[t] : vp.bar, here ? (uint32_t)used[t] & 1 : vp.parity};
            if (QUEUE && here && first[t] && outs[t] > 0) ok = warp_wait(&s.o_empty[t], (outs[t] - 1) & 1, ab);
            if (!ok) break;
            if (!loaded) {
              ok = more ? warp_wait_all(ab, vp, kp, pp) : warp_wait_all(ab, vp, pp);
              loaded = true;
            } else if (here) {
              ok = warp_wait(pp.bar, pp.parity, ab);
            }
            if (!ok) break;
            if (here) {
              tc::tc_fence_after();
              const uint32_t v_lo = desc_lo(s.KV[stage(vp)]);
#pragma unroll
              for (int k = 0; k < TILE / 16; ++k)
                mma_ts(tmem + T_O + t * TILE, tmem + T_S + t * TILE + 8 * k, v_lo + k * (16 * 128 >> 4), id_o, !first[t] || k > 0);
              ++used[t];
              first[t] = false;
              if (j + w.step >= w.r[t].hi) {
                commit(&s.o_full[t]);
                ++outs[t];
              }
            }
            if (more && w.works(t, j + w.step)) score(t, stage(kp));
          }
          if (!ok) break;
          commit(&s.empty[stage(vp)]);
          if (more) commit(&s.empty[stage(kp)]);
          if (QUEUE && j + w.step == j1 - 1) commit(&s.q_empty);  // (the last scores)
        }
      }
      commit(&s.done);
      wait_some(&s.done, 0);
    } else if (warp == 10) {
      if constexpr (QUEUE) {
        BlockFinder<true> finder(a, 2 * tokens);
        s.queue.run(ab, [&](int item) {
          w.find(fa, finder, item);
          return w;
        });
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;\n");
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t ts = lanes + T_S + t * TILE, to = lanes + T_O + t * TILE;
    const float c = a.scale * LOG2E;
    bool ok = true;
    int tiles = 0, outs[2] = {0, 0}, merges = 0;
    while (ok && next_item(false)) {
      const AttnBlock& b = w.b;
      const bool dual = w.dual, other = dual && t == 1;
      const int i0 = b.first + (dual ? 0 : t * tokens), i1 = min(b.lq, i0 + tokens);
      const int token = i0 + (row >> fa.pack), h = w.h0 + (row & (heads - 1));
      const bool live = token < b.lq;
      const KeyRange kr = keys_of(a, token, b.lq, b.lk);
      float m = -INFINITY, l = 0.f;  // the maximum (of scores before the scale), the sum
      const KeyRange seen{keys_of(a, i1 - 1, b.lq, b.lk).lo, keys_of(a, i0, b.lq, b.lk).hi};  // keys every row sees
      bool first = true;
      for (int j = w.r[t].lo + (other ? 1 : 0); j < w.r[t].hi; j += w.step) {
        ok = warp_wait(&s.s_full[t], tiles++ & 1, ab);
        if (!ok) break;
        tc::tc_fence_after();
        uint32_t x[TILE];
#pragma unroll
        for (int i = 0; i < TILE; i += 32) tc::tmem_ld32(ts + i, x + i);
        tc::tmem_wait_ld();
        pin(x);
        if (j * TILE < seen.lo || (j + 1) * TILE > seen.hi) {
          const int lo = kr.lo - j * TILE, hi = kr.hi - j * TILE;
#pragma unroll
          for (int i = 0; i < TILE; ++i) x[i] = i >= lo && i < hi ? x[i] : 0xff800000u;
        }
        float top[4] = {m, m, m, m};
#pragma unroll
        for (int i = 0; i < TILE; ++i) top[i & 3] = fmaxf(top[i & 3], __uint_as_float(x[i]));
        const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        // (and of -inf: the first keys a row sees; rows of the next document do not ask)
        if (__any_sync(0xffffffffu, live && (mx - m) * c > 8.f)) {
          const float f = m == -INFINITY ? 0.f : ex2((m - mx) * c);
          m = mx;
          l *= f;
          if (!first) {  // the products before this tile's scores are complete
#pragma unroll 1
            for (int i = 0; i < DB * 64; i += 32) {
              uint32_t o[32];
              tc::tmem_ld32(to + i, o);
              tc::tmem_wait_ld();
              pin(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tc::tmem_st32(to + i, o);
            }
          }
        }
        first = false;
        const float base = m == -INFINITY ? 0.f : -m * c;
        const uint64_t cc = pack2(c, c), bb = pack2(base, base);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < TILE; i += 2) {
          const uint64_t e = fma2(pack2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), cc, bb);
          float p, q;
          unpack2(e, p, q);
          p = ex2(p);
          q = ex2(q);
          sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], pack2(p, q));
          const __nv_bfloat162 v = __floats2bfloat162_rn(p, q);
          x[i / 2] = *reinterpret_cast<const uint32_t*>(&v);
        }
        tc::tmem_st32(ts, x);
        tc::tmem_st32(ts + 32, x + 32);
        l += sum_of(add2(sum[0], sum[1]));
        tc::tmem_wait_st();
        tc::tc_fence_before();
        warp_arrive(&s.p_full[t]);
      }
      if (!ok) break;
      const int64_t at = (int64_t)(b.q0 + token);
      const bool any = w.any(t);
      if (dual) {
        ok = warp_wait_all(ab, Phase{&s.o_full[0], (uint32_t)outs[0] & 1}, Phase{&s.o_full[1], (uint32_t)outs[1] & 1});
      } else if (any) {
        ok = warp_wait(&s.o_full[t], (t ? outs[1] : outs[0]) & 1, ab);
      }
      if (!ok) break;
      outs[0] += w.any(0);
      outs[1] += w.any(1);
      tc::tc_fence_after();
      // The halves of a dual tile: the second's sums and out cross shared memory (both places of
      // Q, which the products have read) to the first.
      static_assert(TILE * DB * 64 * 4 <= sizeof(s.Q), "a tile of FP32");
      float* swap = reinterpret_cast<float*>(s.Q) + row * DB * 64;
      auto place = [&](int i) { return (i / 4 ^ (row & 15)) * 4; };  // (rows are a multiple of 32 banks apart)
      const bool rows = __any_sync(0xffffffffu, live);
      float f0 = 1.f, f1 = 0.f;
      if (other) {
        s.m[row] = m;
        s.l[row] = l;
        if (rows) {
#pragma unroll 1
          for (int i = 0; i < DB * 64; i += 32) {
            uint32_t o[32];
            tc::tmem_ld32(to + i, o);
            tc::tmem_wait_ld();
            pin(o);
            if (live)
#pragma unroll
              for (int k = 0; k < 32; k += 4) *reinterpret_cast<uint4*>(swap + place(i + k)) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
        }
        tc::tc_fence_before();
        if (QUEUE) warp_arrive(&s.o_empty[1]);
        warp_arrive(&s.merged);
        continue;
      }
      if (dual) {
        ok = warp_wait(&s.merged, merges++ & 1, ab);
        if (!ok) break;
        const float m1 = s.m[row], top = fmaxf(m, m1);
        f0 = m == -INFINITY ? 0.f : ex2((m - top) * c);
        f1 = m1 == -INFINITY ? 0.f : ex2((m1 - top) * c);
        l = fmaf(l, f0, s.l[row] * f1);
        m = top;
      }
      const float f = l == 0.f ? 0.f : 1.f / l;
      f0 *= f;
      f1 *= f;
      __nv_bfloat16* out = a.out + (at * a.H + h) * a.D;
      float* part_out = fa.part_out + ((w.part * a.T + at) * a.H + h) * a.D;
#pragma unroll 1
      for (int i = 0; i < DB * 64 && rows; i += 32) {
        uint32_t o[32];
        if (any) {
          tc::tmem_ld32(to + i, o);
          tc::tmem_wait_ld();
          pin(o);
        }
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = l == 0.f ? 0.f : __uint_as_float(o[k]) * f0;
        if (dual && live)
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float4 x = *reinterpret_cast<const float4*>(swap + place(i + k));
            v[k] = fmaf(x.x, f1, v[k]);
            v[k + 1] = fmaf(x.y, f1, v[k + 1]);
            v[k + 2] = fmaf(x.z, f1, v[k + 2]);
            v[k + 3] = fmaf(x.w, f1, v[k + 3]);
          }
        if (fa.parts > 1) {
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            if (live && i + k < a.D) *reinterpret_cast<float4*>(part_out + i + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
          continue;
        }
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
          uint32_t u[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(v[k + 2 * e], v[k + 2 * e + 1]);
            u[e] = *reinterpret_cast<const uint32_t*>(&x);
          }
          if (live && i + k < a.D) *reinterpret_cast<uint4*>(out + i + k) = make_uint4(u[0], u[1], u[2], u[3]);
        }
      }
      if (QUEUE && any) {
        tc::tc_fence_before();
        warp_arrive(&s.o_empty[t]);
      }
      if (QUEUE && dual) {
        tc::fence_proxy_async();  // (Q comes by asynchronous copies again)
        warp_arrive(&s.swapped);
      }
      float* lse = fa.parts > 1 ? fa.part_lse + (int64_t)w.part * a.H * a.T : a.lse;
      if (live) lse[h * a.T + at] = l == 0.f ? -INFINITY : (m * c + log2f(l)) * 0.69314718f;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && s.abort) atomicExch(fa.err, 11);
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// The parts of a query's keys joined: lse = log sum e^lse_p, out = sum e^(lse_p - lse)
// out_p.  A warp a query and head.
__global__ void __launch_bounds__(256) k_attn_join(const __grid_constant__ FwdArgs fa) {
  const AttnArgs& a = fa.a;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  previous_ended();
  if (row >= a.T * a.H) return;
  const int64_t t = row / a.H, at = row % a.H * a.T + t, stride = a.T * a.H;
  float top = -INFINITY;
  bool none = true;  // (a part of nothing but NaN has seen keys)
  for (int p = 0; p < fa.parts; ++p) {
    const float l = fa.part_lse[p * stride + at];
    top = fmaxf(top, l);
    none = none && l == -INFINITY;
  }
  float sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = 0; p < fa.parts && !none; ++p) {
    const float w = ex2((fa.part_lse[p * stride + at] - top) * LOG2E);
    sum += w;
    if (4 * lane < a.D) {
      const float4 x = *reinterpret_cast<const float4*>(fa.part_out + (p * stride + row) * a.D + 4 * lane);
      o.x = fmaf(w, x.x, o.x);
      o.y = fmaf(w, x.y, o.y);
      o.z = fmaf(w, x.z, o.z);
      o.w = fmaf(w, x.w, o.w);
    }
  }
  const float f = none ? 0.f : 1.f / sum;
  if (4 * lane < a.D) {
    const float v[4] = {o.x * f, o.y * f, o.z * f, o.w * f};
    vstore<__nv_bfloat16, 4>(a.out + row * a.D + 4 * lane, v);
  }
  if (lane == 0) a.lse[at] = none ? -INFINITY : top + logf(sum);
}

}  // namespace

cudaError_t launch_attn_fwd(const AttnArgs& a, const AttnPlan& p, const int32_t* cu, const int32_t* cuk, float* scratch,
                            cudaStream_t st) {
  FwdArgs f{};
  f.a = a;
  f.err = device_error_ptr();
  if (!f.err) return cudaErrorUnknown;
  f.pack = p.pack;
  f.parts = p.fwd;
  f.part_out = scratch;
  f.part_lse = scratch + (int64_t)p.fwd * a.T * a.H * a.D;
  const int per = 2 * (TILE >> f.pack);
  int64_t blocks = 0;
  for (int i = 0; i < a.N; ++i) blocks += (cu[i + 1] - cu[i] + per - 1) / per;
  if (!attn_map(&f.q_map, a.q, a.T, a.H, a.D, 1 << f.pack, TILE >> f.pack)) return cudaErrorInvalidValue;
  if (a.TK > 0 && (!attn_map(&f.k_map, a.k, a.TK, a.HK, a.D, 1, TILE) || !attn_map(&f.v_map, a.v, a.TK, a.HK, a.D, 1, TILE)))
    return cudaErrorInvalidValue;
  blocks *= (a.H >> f.pack) * f.parts;
  const int64_t rows = (a.T * a.H + 7) / 8;
  if (blocks > INT32_MAX || rows > INT32_MAX) return cudaErrorInvalidValue;
  if (blocks > sm_count()) attn_order(f.a, cuk);
  auto go = [&](auto kernel, size_t smem) {
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) return e;
    return launch_early(kernel, dim3((unsigned)blocks), THREADS, smem, st, f);
  };
  static_assert(sizeof(FwdSmem<1>) <= 232448 && sizeof(FwdSmem<2>) <= 232448, "227 KB of shared memory a block");
  // Blocks that take over others' items gain on short ones of up to 64 columns, whose start and end
  // they hide: 16384 tokens of 16 heads, windows of 128 / 1024 / 4096: 71 / 135 / 316 us against 82 /
  // 142 / 319; of 128 columns they lose (98 / 175 / 403 against 98 / 169 / 385).
  {
    ProfScope ps("attn_fwd", st, (double)a.T * a.H);
    if (cudaError_t e = a.D > 64                 ? go(k_attn_fwd<2, false>, sizeof(FwdSmem<2>))
                        : blocks <= sm_count() ? go(k_attn_fwd<1, false>, sizeof(FwdSmem<1>))
                                               : go(k_attn_fwd<1, true>, sizeof(FwdSmem<1>)))
      return e;
  }
  if (f.parts == 1) return cudaSuccess;
  ProfScope ps("attn_join", st, (double)a.T * a.H);
  return launch_early(k_attn_join, dim3((unsigned)rows), 256, 0, st, f);
}

// Heads that share their keys lie side by side while the longest document's queries alone do
// not fill a tile.
//
// Parts: few blocks, or few of them much longer than the rest, leave SMs without work.  The
// number with the least estimated time is taken, in steps of a block (two tiles' products,
// some 1.4 us): a block's start and end, with the share that it leaves where there are
// several, and the join's traffic.  Measured in 1 / 2 / 3 / 4 / 8 parts, the join's time
// included: one token of 65536 keys, 8 key heads 520 / 272 / 190 / 146 / 88 us, 16 parts 73; a
// prompt of 24576 tokens of one head 319 / 180 / 137 / 156 / 181; dK and dV of 4096 tokens, 16
// heads over 4 key heads 178 / 109 / 129 / 132 / 179; 80 to 160 single tokens of 8 key heads, one of 65536 keys,
// the others of 1000, 528 / 272.  The number is one for the call: cutting the short documents as well costs
// their blocks' starts, which of 256 such tokens is as much as it gains (537 us in one part).  Packs of more
// than 1024 tiles of rows are not looked at, for the host's time (up to there 20 us).  152 SMs: the
// sizes of workspaces are the same without a GPU.
AttnPlan attn_plan(const AttnArgs& a, const int32_t* cu, const int32_t* cuk) {
  AttnPlan p{0, 1, 1, 1, 0, 0};
  int most = 0;
  for (int i = 0; i < a.N; ++i) most = std::max(most, cu[i + 1] - cu[i]);
  const int G = a.H / a.HK;
  while (p.pack < 7 && G % (2 << p.pack) == 0 && ((int64_t)most << p.pack) < TILE) ++p.pack;
  const double sms = 152.0, kStart = 4.0, kShare = 4.0, kJoin = 2.0, kBytes = 8e6;  // (bytes that HBM moves in a step)
  const int tokens = TILE >> p.pack;
  // parts of blocks of `per` rows of `lens`, `heads` a block each, `rows` of FP32 left by a part
  auto parts = [&](const int32_t* lens, int per, int64_t heads, double row_bytes, auto tiles) {
    int64_t blocks = 0;
    for (int i = 0; i < a.N; ++i) blocks += (lens[i + 1] - lens[i] + per - 1) / per;
    if (blocks == 0 || blocks > 1024) return 1;
    blocks *= heads;
    int64_t total = 0, longest = 0;
    for (int i = 0; i < a.N; ++i)
      for (int at = 0; at < lens[i + 1] - lens[i]; at += per) {
        const int64_t n = tiles(cu[i + 1] - cu[i], cuk[i + 1] - cuk[i], at);
        total += n * heads;
        longest = std::max(longest, n);
      }
    int best = 1;
    double least = 0;
    for (int s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
      if (s > 1 && s > longest / 2) break;
      const double start = kStart + (s > 1 ? kShare : 0.0);
      double time = std::max((double)((longest + s - 1) / s) + start, (total + start * blocks * s) / sms);
      if (s > 1) time += kJoin + 2.0 * s * row_bytes / kBytes;
      if (s == 1 || time < 0.9 * least) {
        best = s;
        least = time;
      }
    }
    return best;
  };
  const double out_bytes = 4.0 * a.T * a.H * a.D, key_bytes = 8.0 * a.TK * a.HK * a.D;
  p.fwd = parts(cu, 2 * tokens, a.H >> p.pack, out_bytes, [&](int lq, int lk, int at) {
    const TileRange r = tiles_of(a, lq, lk, at, std::min(lq, at + 2 * tokens));
    const int n = r.hi - r.lo;
    return at + tokens >= lq ? (n + 1) / 2 : n;  // (two key tiles a step where the second tile has no queries)
  });
  p.dq = parts(cu, tokens, a.H >> p.pack, out_bytes, [&](int lq, int lk, int at) {
    const TileRange r = tiles_of(a, lq, lk, at, std::min(lq, at + tokens));
    return r.hi - r.lo;
  });
  p.dkv = parts(cuk, TILE, a.HK, key_bytes, [&](int lq, int lk, int at) {
    const TileRange r = query_tiles_of(a, lq, lk, at, std::min(lk, at + TILE) - 1, tokens);
    return (r.hi - r.lo) * (G >> p.pack);
  });
  auto floats = [](int parts, double n) { return parts > 1 ? (size_t)parts * (size_t)n * sizeof(float) : 0; };
  const size_t rows = (size_t)a.T * a.H;
  p.fwd_bytes = floats(p.fwd, (double)rows * (a.D + 1));
  p.bwd_bytes = std::max(floats(p.dq, (double)rows * (a.D + 4)), floats(p.dkv, 2.0 * a.TK * a.HK * a.D));
  return p;
}

bool attn_tc_shape(int D) { return D % 8 == 0 && D <= 128; }

}  // namespace gdr
