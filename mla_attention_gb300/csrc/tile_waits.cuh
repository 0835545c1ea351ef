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

// D (+)= A B over a 64-column box of 16-bit values: four K16 steps along 128-byte swizzled rows of both operands
__device__ __forceinline__ void mma_box64(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 t, %3, %3;\n\tmov.b64 x, %1;\n\tmov.b64 y, %2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\tadd.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\tadd.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\tadd.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

}  // namespace mla
