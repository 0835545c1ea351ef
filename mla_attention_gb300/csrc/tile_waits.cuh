// Bounded waits of the kernels over a smaller cache.  A wait that runs out sets the CTA's abort word, which ends the other
// waits of the CTA, and records its site in the call's status word.  Range codes of earlier calls in that word end nothing.
#pragma once
#include "sm103_ptx.cuh"

namespace mla {

// The part of a wait behind its first test, out of line: a kernel has dozens of waits, and its loops should stay in the
// instruction cache.
static __device__ __noinline__ bool tile_wait_on(uint64_t* bar, uint32_t parity, uint32_t* abort, uint32_t* err, uint32_t site,
                                                 uint32_t spin_limit, bool cluster) {
  if (mbar_wait_inline(bar, parity, abort, site, spin_limit, cluster)) return true;
  atomicCAS(abort, 0u, DEV_TIMEOUT_BASE | site);
  record_error(err, DEV_TIMEOUT_BASE | site);
  return false;
}

struct TileWaits {
  uint32_t* abort;     // shared memory, 0 at the start
  uint32_t* err;       // the call's status word
  uint32_t spin_limit;

  // by a warp, with one answer for all of it
  __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity, uint32_t site, bool cluster = false) const {
    const uint32_t a = smem_u32(bar);
    if (__all_sync(0xffffffffu, cluster ? mbar_try_wait_cluster(a, parity) : mbar_try_wait(a, parity))) return true;
    const bool ok = tile_wait_on(bar, parity, abort, err, site, spin_limit, cluster);
    return __all_sync(0xffffffffu, ok);
  }
};

// One arrival for the warp on a barrier of the first CTA, whose warps then issue MMAs over both CTAs' memory.  kShared: what it tells of
// are writes to this CTA's own shared memory, released to the cluster by a fence that is restricted to them; else uses of
// tensor memory, which the tcgen05 fences before the arrival and behind the wait order.  (An arrival that releases everything
// waits for the loads on their way: 64 requests of the 4-bit decode 479 us for 352, 4096 rows of the key weights 146 for 126.)
template <bool kShared>
__device__ __forceinline__ void first_cta_arrive(uint64_t* bar, uint32_t cta) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    if (cta == 0) mbar_arrive(bar);
    else {
      if (kShared) asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
      asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_to_rank(smem_u32(bar), 0)) : "memory");
    }
  }
}
// arrives on the barrier once the MMAs that this thread issued are done; of a pair, at this offset in both CTAs
template <int kCtas>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (kCtas == 1) mma_commit(bar);
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
               "h"((uint16_t)3)
               : "memory");
}

#define MLA_BOX64(G, P) "tcgen05.mma.cta_group::" G ".kind::f16 [%0], x, y, %3, " P ";\n\t"
#define MLA_BOX64_4(G) \
  "{\n\t.reg .pred p, t;\n\t.reg .b64 x, y;\n\t" \
  "setp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 t, %3, %3;\n\tmov.b64 x, %1;\n\tmov.b64 y, %2;\n\t" \
  MLA_BOX64(G, "p") "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t" MLA_BOX64(G, "t") "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t" \
  MLA_BOX64(G, "t") "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t" MLA_BOX64(G, "t") "}"
// D (+)= A B over a 64-column box of 16-bit values: four K16 steps along 128-byte swizzled rows of both operands
template <int kCtas>
__device__ __forceinline__ void mma_box64(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kCtas == 1) asm volatile(MLA_BOX64_4("1") ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
  else asm volatile(MLA_BOX64_4("2") ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
#undef MLA_BOX64
#undef MLA_BOX64_4

}  // namespace mla
