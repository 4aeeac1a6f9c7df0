// gdr_attn_tc.cuh -- pieces of the attention kernels on the tensor cores.
#pragma once
#include <algorithm>

#include "gdr_attn.cuh"
#include "gdr_tc_roles.cuh"

namespace gdr {

constexpr int TILE = 128;  // rows of a tile of queries or keys

// The tiles [lo, hi) that a block goes through.
struct TileRange {
  int lo, hi;
};
// Of keys: those that queries [i0, i1) of a document see.
__host__ __device__ __forceinline__ TileRange tiles_of(const AttnArgs& a, int lq, int lk, int i0, int i1) {
  if (i0 >= i1) return {0, 0};
  const KeyRange first = keys_of(a, i0, lq, lk), last = keys_of(a, i1 - 1, lq, lk);
  if (last.hi <= first.lo) return {0, 0};
  return {first.lo / TILE, (last.hi + TILE - 1) / TILE};
}
// Of queries, `tokens` a tile: those that see any of the keys [first, last].
__host__ __device__ __forceinline__ TileRange query_tiles_of(const AttnArgs& a, int lq, int lk, int first, int last, int tokens) {
  const int off = lk - lq;
  const int lo = a.causal && first > off ? first - off : 0;
  int hi = lq;
  if (a.window && (int64_t)last - off + a.window < lq) hi = last - off + a.window;
  if (hi <= lo) return {0, 0};
  return {lo / tokens, (hi + tokens - 1) / tokens};
}
// Part `part` of `parts` of a range.
__device__ __forceinline__ TileRange part_of(const TileRange& r, int part, int parts) {
  const int64_t n = r.hi - r.lo;
  return {r.lo + (int)(n * part / parts), r.lo + (int)(n * (part + 1) / parts)};
}

template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N]) {  // nothing that reads them moves before this
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// The items that a block works on, its own first and then those of blocks that have not
// begun, which it takes over (cluster launch control): what starts and ends a block
// overlaps between its items, and the longest items still come first.  One warp asks for
// items and forms what the others need of them: each of them doing so for itself took some
// 3500 clocks an item, of instructions fetched for the one use.
template <typename Work>
struct WorkQueue {
  alignas(16) uint4 answer;
  alignas(16) Work work[2];
  int more[2];
  uint64_t full[2], empty[2], wanted, asked;

  __device__ __forceinline__ void init(int takers) {  // (one thread; warps that take)
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], takers);
    }
    tc::mbar_init(&wanted, 1);
    tc::mbar_init(&asked, 1);
  }
  // The warp that asks: make(item) -> Work.  The others ask for the next item when they have
  // gone through all steps of the last, each of which has waits of its own limit.
  template <typename F>
  __device__ __forceinline__ void run(volatile int* abort, F make) {
    const int lane = threadIdx.x & 31;
    int item = (int)blockIdx.x;
    bool have = true;
    ByClock limit;
    for (int k = 0;; ++k) {
      const int e = k & 1;
      if (k >= 2 && !warp_wait(&empty[e], ((k >> 1) - 1) & 1, abort)) return;
      if (have) {
        const Work w = make(item);
        limit.ns = kWaitNs * (1 + (uint64_t)w.steps());
        if (lane == 0) work[e] = w;
      }
      if (lane == 0) more[e] = have;
      warp_arrive(&full[e]);
      if (!have || !warp_wait_within(limit, abort, Phase{&wanted, (uint32_t)e})) return;
      if (lane == 0) {
        tc::fence_proxy_async();  // (the last answer has been read)
        tc::mbar_arrive_expect_tx(&asked, 16);
        asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(
                         tc::smem_u32(&answer)),
                     "r"(tc::smem_u32(&asked))
                     : "memory");
      }
      __syncwarp();
      if (!warp_wait(&asked, e, abort)) {
        wait_some(&asked, e);
        return;
      }
      uint32_t taken, next;
      asm volatile(
          "{\n .reg .pred p;\n .reg .b128 r;\n .reg .b64 lo, hi;\n ld.shared.v2.b64 {lo, hi}, [%2];\n mov.b128 r, {lo, hi};\n"
          " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
          " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}\n"
          : "=r"(taken), "=r"(next)
          : "r"(tc::smem_u32(&answer))
          : "memory");
      have = __shfl_sync(0xffffffffu, taken, 0) != 0;
      item = (int)__shfl_sync(0xffffffffu, next, 0);
    }
  }
  // The same of those of every gridDim-th item that are to be done: of the first n as known[] has
  // it, of the others as pick(work) answers.
  template <typename F, typename P>
  __device__ __forceinline__ void run_those(volatile int* abort, int items, F make, const uint8_t* known, int n, P pick) {
    const int lane = threadIdx.x & 31;
    ByClock limit;
    int k = 0;
    for (int64_t i = 0;; ++i) {
      const int64_t item = blockIdx.x + i * gridDim.x;
      const bool have = item < items;
      Work w;
      if (have) {
        if (i < n && !known[i]) continue;
        w = make((int)item);
        if (i >= n && !pick(w)) continue;
      }
      const int e = k & 1;
      if (k >= 1 && !warp_wait_within(limit, abort, Phase{&wanted, (uint32_t)e ^ 1})) return;
      if (k >= 2 && !warp_wait(&empty[e], ((k >> 1) - 1) & 1, abort)) return;
      if (lane == 0) {
        if (have) work[e] = w;
        more[e] = have;
      }
      warp_arrive(&full[e]);
      if (!have) return;
      limit.ns = kWaitNs * (1 + (uint64_t)w.steps());
      ++k;
    }
  }
  // A taking warp's next item, its k-th; false: there is none.  The warp that loads asks for
  // it, when all loads of the last one are on their way: a block that asked sooner would hold
  // items that others have nothing to do for.
  __device__ __forceinline__ bool take(int& k, Work& w, volatile int* abort, bool ask) {
    const int e = k & 1;
    if (ask && k > 0) warp_arrive(&wanted);
    if (!warp_wait(&full[e], (k >> 1) & 1, abort)) return false;
    const bool is = more[e];
    if (is) w = work[e];
    warp_arrive(&empty[e]);
    ++k;
    return is;
  }
};

// Whether TMA addresses the tensors.
inline bool attn_tc_layout(const AttnArgs& a) {
  for (const AttnRows* t : {&a.q, &a.k, &a.v, &a.dout})
    if (t->p && (((uintptr_t)t->p & 15) != 0 || t->s0 <= 0 || t->s1 <= 0 || t->s0 % 8 != 0 || t->s1 % 8 != 0 ||
                 std::max(t->s0, t->s1) >= (int64_t)1 << 39))
      return false;
  for (const void* p : {(const void*)a.out, (const void*)a.o, (const void*)a.dq, (const void*)a.dk, (const void*)a.dv})
    if (((uintptr_t)p & 15) != 0) return false;
  return true;
}

// Orders the documents for blocks that do not all run at a time.
inline void attn_order(AttnArgs& a, const int32_t* cuk) {
  a.ordered = a.N > 1 && a.N <= ATTN_ORDERED;
  if (!a.ordered) return;
  for (int i = 0; i < a.N; ++i) a.order[i] = (uint8_t)i;
  auto keys = [&](int i) { return cuk[i + 1] - cuk[i]; };
  std::sort(a.order, a.order + a.N, [&](int x, int y) { return keys(x) != keys(y) ? keys(x) > keys(y) : x < y; });
}

// [T][heads][D] BF16: boxes of 64 elements x `heads` heads x `tokens` tokens, 128-byte
// swizzle, zero fill outside.
inline bool attn_map(CUtensorMap* map, const AttnRows& t, int64_t T, int H, int D, int heads, int tokens) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  cuuint64_t strides[2] = {(cuuint64_t)t.s1 * 2, (cuuint64_t)t.s0 * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(t.p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gdr
