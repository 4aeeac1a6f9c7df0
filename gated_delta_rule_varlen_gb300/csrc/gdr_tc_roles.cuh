// gdr_tc_roles.cuh -- pieces of kernels whose warps play roles around tcgen05 products:
// bounded waits that let a whole block give up together, products and commits issued
// by one elected thread of a converged warp, and the tensor map encoder.  Operand tiles
// are blocks of 128 rows of 64 BF16 (128 bytes), swizzled, side by side.
#pragma once
#include <cudaTypedefs.h>

#include "gdr_ops.cuh"
#include "gdr_tc.cuh"

namespace gdr {

constexpr int BLK = 128 * 128;  // bytes of a tile block: 128 rows of 64 BF16

// Waits of the blocks' roles.  Each gives up when its limit is over, or once another role has,
// and returns false; the block then reports the timeout as it ends.  Few instructions: the
// roles run straight through long loops that share the instruction cache.
constexpr uint64_t kWaitNs = 2000000000ull;
// A limit by the clock, read every sixteenth try; a try is suspended until the phase completes or
// the hardware's own limit passes (with a limit of a microsecond asked for, the attention kernels
// took 3 to 4% longer).
struct ByClock {
  static constexpr uint32_t SUSPEND = 0;
  uint64_t ns = kWaitNs, start = 0;
  __device__ __forceinline__ bool over(int tries) {
    if ((tries & 15) != 15) return false;
    const uint64_t now = tc::global_ns();
    if (start == 0) start = now;
    return now - start > ns;
  }
};
// 2^20 tries of at most a microsecond: the fewest instructions (the scan of 32768 tokens takes
// 441 us, with the clock 466).
struct ByTries {
  static constexpr uint32_t SUSPEND = 1000;
  __device__ __forceinline__ bool over(int tries) { return tries > 1 << 20; }
};
template <typename Limit>
__device__ __forceinline__ bool try_phase(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  if constexpr (Limit::SUSPEND > 0)
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(tc::smem_u32(bar)), "r"(parity), "r"(Limit::SUSPEND)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
  return done != 0;
}
template <typename Limit>
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort) {
  Limit limit;
  for (int tries = 0; !try_phase<Limit>(bar, parity); ++tries)
    if (limit.over(tries) || *abort) {
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
// Asks for a tensor map, which the first copy would wait for.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// One arrival for the warp, after all its lanes' work.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive(bar);
}
// The wait of a whole warp for one or several barriers: the same answer on every lane.  A wait
// costs some 200 clocks even where its phase is complete, several together that once.
struct Phase {
  uint64_t* bar;
  uint32_t parity;
};
template <typename Limit, typename... P>
__device__ __forceinline__ bool warp_wait_within(Limit limit, volatile int* abort, P... p) {
  for (int tries = 0; !__all_sync(0xffffffffu, (try_phase<Limit>(p.bar, p.parity) & ...)); ++tries)
    if (__any_sync(0xffffffffu, limit.over(tries) || *abort)) {
      *abort = 1;
      return false;
    }
  return true;
}
template <typename Limit = ByClock, typename... P>
__device__ __forceinline__ bool warp_wait_all(volatile int* abort, P... p) {
  return warp_wait_within(Limit{}, abort, p...);
}
template <typename Limit = ByClock>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return warp_wait_all<Limit>(abort, Phase{bar, parity});
}
// A wait before a block ends, whatever has happened: 20 ms at most, and what a try is
// suspended for.
__device__ __forceinline__ void wait_some(uint64_t* bar, uint32_t parity) {
  if (try_phase<ByClock>(bar, parity)) return;
  const uint64_t start = tc::global_ns();
  while (!try_phase<ByClock>(bar, parity) && tc::global_ns() - start < 20000000ull) {
  }
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

inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
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

}  // namespace gdr
