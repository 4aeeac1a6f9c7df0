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
// needs): 2^-9 of each term at most, independently.
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
  int* err;
};

constexpr int THREADS = 384;
// Tensor memory: S (and over it P) of the tiles, out of the tiles.
constexpr int T_S = 0, T_O = 256;

template <int DB>  // blocks of 64 columns
struct FwdSmem {
  static constexpr int STAGES = DB == 2 ? 5 : 10;
  unsigned char Q[2][DB * BLK];
  unsigned char KV[STAGES][DB * BLK];  // K and V tiles in turn
  uint64_t q_full[2], full[STAGES], empty[STAGES], cleared;
  uint64_t s_full[2], p_full[2], o_full[2], done;
  uint32_t tmem;
  int abort;
};

template <int DB>
__global__ void __launch_bounds__(THREADS, 1) k_attn_fwd(const __grid_constant__ FwdArgs fa) {
  using Smem = FwdSmem<DB>;
  constexpr int ST = Smem::STAGES;
  extern __shared__ unsigned char attn_smem[];
  Smem& s = *reinterpret_cast<Smem*>(tc::align1024(attn_smem));
  const AttnArgs& a = fa.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* ab = &s.abort;
  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        tc::mbar_init(&s.q_full[i], 1);
        tc::mbar_init(&s.s_full[i], 1);
        tc::mbar_init(&s.p_full[i], 4);
        tc::mbar_init(&s.o_full[i], 1);
      }
      for (int i = 0; i < ST; ++i) {
        tc::mbar_init(&s.full[i], 1);
        tc::mbar_init(&s.empty[i], 1);
      }
      tc::mbar_init(&s.cleared, 1);
      tc::mbar_init(&s.done, 1);
      s.abort = 0;
      tc::mbar_fence_init();
    }
    __syncwarp();
    tc::tmem_alloc(&s.tmem, 512);
    tc::tmem_relinquish();
  }
  const int heads = 1 << fa.pack, tokens = TILE >> fa.pack;  // of a tile
  const int groups = a.H >> fa.pack;
  const AttnBlock b = find_block<true>(a, a.cu, 2 * tokens, blockIdx.x / groups);
  const int h0 = (int)(blockIdx.x % groups) * heads, hk = h0 / (a.H / a.HK);
  TileRange r[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int i0 = b.first + t * tokens;
    r[t] = tiles_of(a, b, i0, min(b.lq, i0 + tokens));
  }
  // (an empty range follows the other one)
  if (r[0].lo >= r[0].hi) r[0].lo = r[0].hi = r[1].lo;
  if (r[1].lo >= r[1].hi) r[1].lo = r[1].hi = r[0].hi;
  const int j0 = min(r[0].lo, r[1].lo), j1 = max(r[0].hi, r[1].hi);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s.tmem;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
    if (warp == 8 && j0 < j1) {  // loads
      if (lane == 0)
        for (int t = 0; t < 2; ++t)
          if (r[t].lo < r[t].hi) {
            tc::mbar_arrive_expect_tx(&s.q_full[t], DB * BLK);
            for (int c = 0; c < DB; ++c)
              tc::tma_load_3d(s.Q[t] + c * BLK, &fa.q_map, 64 * c, h0, b.q0 + b.first + t * tokens, &s.q_full[t]);
          }
      __syncwarp();
      const int n = 2 * (j1 - j0);
      int i = 0;
      for (int st = 0, ph = 0; i < n; ++i) {
        const int j = j0 + (i >> 1);
        const bool isv = i & 1;
        if (i >= ST && !warp_wait(&s.empty[st], ph ^ 1, ab)) break;
        const int rows = b.lk - j * TILE;
        uint64_t* bar = isv && rows < TILE ? &s.cleared : &s.full[st];
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(bar, DB * BLK);
          for (int c = 0; c < DB; ++c)
            tc::tma_load_3d(s.KV[st] + c * BLK, isv ? &fa.v_map : &fa.k_map, 64 * c, hk, b.k0 + j * TILE, bar);
        }
        __syncwarp();
        if (isv && rows < TILE) {  // the document's last tile: clear what lies behind it
          if (!warp_wait(&s.cleared, 0, ab)) break;
          for (int e = rows * 8 + lane; e < TILE * 8; e += 32)
            for (int c = 0; c < DB; ++c) *reinterpret_cast<uint4*>(s.KV[st] + c * BLK + e * 16) = make_uint4(0, 0, 0, 0);
          tc::fence_proxy_async();
          warp_arrive(&s.full[st]);
        }
        if (++st == ST) {
          st = 0;
          ph ^= 1;
        }
      }
      if (i < n) {  // given up: the copies in flight land before the block ends
        for (int k = max(0, i - ST); k < i; ++k) wait_some(&s.full[k % ST], (k / ST) & 1);
        for (int t = 0; t < 2; ++t)
          if (r[t].lo < r[t].hi) wait_some(&s.q_full[t], 0);
      }
    } else if (warp == 9 && j0 < j1) {  // products
      const uint32_t id_s = tc::idesc_bf16(TILE, TILE);
      const uint32_t id_o = tc::idesc_bf16(TILE, (a.D + 15) / 16 * 16) | tc::kIdescTransposeB;
      const int ks = (a.D + 15) / 16;
      uint32_t q_lo[2] = {desc_lo(s.Q[0]), desc_lo(s.Q[1])};
      auto score = [&](int t, int st) {
        const uint32_t k_lo = desc_lo(s.KV[st]);
#pragma unroll
        for (int k = 0; k < 4 * DB; ++k) {
          const uint32_t at = ((k >> 2) * BLK + (k & 3) * 32) >> 4;
          if (k < ks) mma_ss(tmem + T_S + t * TILE, q_lo[t] + at, k_lo + at, id_s, k > 0);
        }
        commit(&s.s_full[t]);
      };
      bool ok = true;
      int used[2] = {0, 0};
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
      Phase kp = next();
      ok = warp_wait(kp.bar, kp.parity, ab);
      for (int t = 0; t < 2 && ok; ++t)
        if (r[t].lo < r[t].hi) {
          ok = warp_wait(&s.q_full[t], 0, ab);
          if (ok && r[t].lo == j0) score(t, stage(kp));
        }
      if (ok) commit(&s.empty[stage(kp)]);
      for (int j = j0; j < j1 && ok; ++j) {
        const bool more = j + 1 < j1;
        const Phase vp = next();
        if (more) kp = next();
        bool loaded = false;  // V of this step, K of the next
        for (int t = 0; t < 2 && ok; ++t) {
          const bool here = j >= r[t].lo && j < r[t].hi;
          const Phase pp{here ? &s.p_full[t] : kp.bar, here ? (uint32_t)used[t] & 1 : kp.parity};
          if (!loaded) {
            ok = more ? warp_wait_all(ab, vp, kp, here ? pp : kp) : warp_wait_all(ab, vp, here ? pp : vp);
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
              mma_ts(tmem + T_O + t * TILE, tmem + T_S + t * TILE + 8 * k, v_lo + k * (16 * 128 >> 4), id_o, used[t] > 0 || k > 0);
            ++used[t];
            if (j + 1 == r[t].hi) commit(&s.o_full[t]);
          }
          if (more && j + 1 >= r[t].lo && j + 1 < r[t].hi) score(t, stage(kp));
        }
        if (!ok) break;
        commit(&s.empty[stage(vp)]);
        if (more) commit(&s.empty[stage(kp)]);
      }
      commit(&s.done);
      wait_some(&s.done, 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;\n");
    const int t = warp >> 2, row = tid & 127;
    const int token = b.first + t * tokens + (row >> fa.pack), h = h0 + (row & (heads - 1));
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t ts = lanes + T_S + t * TILE, to = lanes + T_O + t * TILE;
    const bool live = token < b.lq;
    const KeyRange kr = keys_of(a, token, b.lq, b.lk);
    const float c = a.scale * LOG2E;
    float m = -INFINITY, l = 0.f;  // the maximum (of scores before the scale), the sum
    const int i0 = b.first + t * tokens, i1 = min(b.lq, i0 + tokens);
    const KeyRange all{keys_of(a, i1 - 1, b.lq, b.lk).lo, keys_of(a, i0, b.lq, b.lk).hi};  // keys every row sees
    bool ok = true;
    for (int j = r[t].lo, n = 0; j < r[t].hi; ++j, ++n) {
      ok = warp_wait(&s.s_full[t], n & 1, ab);
      if (!ok) break;
      tc::tc_fence_after();
      uint32_t x[TILE];
#pragma unroll
      for (int i = 0; i < TILE; i += 32) tc::tmem_ld32(ts + i, x + i);
      tc::tmem_wait_ld();
      pin(x);
      if (j * TILE < all.lo || (j + 1) * TILE > all.hi) {
        const int lo = kr.lo - j * TILE, hi = kr.hi - j * TILE;
#pragma unroll
        for (int i = 0; i < TILE; ++i) x[i] = i >= lo && i < hi ? x[i] : 0xff800000u;
      }
      float top[4] = {m, m, m, m};
#pragma unroll
      for (int i = 0; i < TILE; ++i) top[i & 3] = fmaxf(top[i & 3], __uint_as_float(x[i]));
      const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      if (__any_sync(0xffffffffu, (mx - m) * c > 8.f)) {  // (and of -inf: the first keys a row sees)
        const float f = m == -INFINITY ? 0.f : ex2((m - mx) * c);
        m = mx;
        l *= f;
        if (n > 0) {  // the products before this tile's scores are complete
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
        const __nv_bfloat162 w = __floats2bfloat162_rn(p, q);
        x[i / 2] = *reinterpret_cast<const uint32_t*>(&w);
      }
      tc::tmem_st32(ts, x);
      tc::tmem_st32(ts + 32, x + 32);
      l += sum_of(add2(sum[0], sum[1]));
      tc::tmem_wait_st();
      tc::tc_fence_before();
      warp_arrive(&s.p_full[t]);
    }
    const int64_t at = (int64_t)(b.q0 + token);
    const bool any = r[t].lo < r[t].hi;
    if (ok && any) {
      ok = warp_wait(&s.o_full[t], 0, ab);
      tc::tc_fence_after();
    }
    if (ok) {
      const float f = l == 0.f ? 0.f : 1.f / l;
      __nv_bfloat16* out = a.out + (at * a.H + h) * a.D;
#pragma unroll 1
      for (int i = 0; i < DB * 64; i += 32) {
        uint32_t o[32];
        if (any) {
          tc::tmem_ld32(to + i, o);
          tc::tmem_wait_ld();
          pin(o);
        }
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(l == 0.f ? 0.f : __uint_as_float(o[k + 2 * e]) * f,
                                                           l == 0.f ? 0.f : __uint_as_float(o[k + 2 * e + 1]) * f);
            w[e] = *reinterpret_cast<const uint32_t*>(&v);
          }
          if (live && i + k < a.D) *reinterpret_cast<uint4*>(out + i + k) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (live) a.lse[h * a.T + at] = l == 0.f ? -INFINITY : (m * c + log2f(l)) * 0.69314718f;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && s.abort) atomicExch(fa.err, 11);
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_attn_fwd(const AttnArgs& a, const int32_t* cu, const int32_t* cuk, cudaStream_t st) {
  FwdArgs f{};
  f.a = a;
  f.err = device_error_ptr();
  if (!f.err) return cudaErrorUnknown;
  f.pack = attn_pack(a, cu);
  const int per = 2 * (TILE >> f.pack);
  int64_t blocks = 0;
  for (int i = 0; i < a.N; ++i) blocks += (cu[i + 1] - cu[i] + per - 1) / per;
  if (!attn_map(&f.q_map, a.q, a.T, a.H, a.D, 1 << f.pack, TILE >> f.pack)) return cudaErrorInvalidValue;
  if (a.TK > 0 && (!attn_map(&f.k_map, a.k, a.TK, a.HK, a.D, 1, TILE) || !attn_map(&f.v_map, a.v, a.TK, a.HK, a.D, 1, TILE)))
    return cudaErrorInvalidValue;
  blocks *= a.H >> f.pack;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  auto go = [&](auto kernel, size_t smem) {
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) return e;
    kernel<<<(unsigned)blocks, THREADS, smem, st>>>(f);
    return cudaGetLastError();
  };
  static_assert(sizeof(FwdSmem<1>) + 1024 <= 232448 && sizeof(FwdSmem<2>) + 1024 <= 232448, "227 KB of shared memory a block");
  ProfScope ps("attn_fwd", st, (double)a.T * a.H);
  return a.D <= 64 ? go(k_attn_fwd<1>, sizeof(FwdSmem<1>) + 1024) : go(k_attn_fwd<2>, sizeof(FwdSmem<2>) + 1024);
}

}  // namespace gdr
