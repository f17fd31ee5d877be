// mx_tile.h -- what the two tiled MXFP4 product kernels share: direct global -> LDS loads of
// whole cache lines, several to one LDS address.
#pragma once
#include "mx_common.h"

namespace nvfp4 {

constexpr int kRow = 128;               // code bytes of a row and stage: 256 elements of K, a cache line
// How early a code descriptor starts: a load's instruction offset (up to 3072) counts for its
// LDS address and its global one, and is taken off the latter again by a scalar that stays
// positive this way.
constexpr uint32_t kBias = 3072;

// dma16 in two: M0, and a load at an offset that moves both its addresses.  Several loads rely on one
// set_m0, so nothing that the compiler makes of these kernels may write M0 in between; a test looks
// through their code for it.  (Taking M0's content from set_m0 into each load as an operand would let
// the compiler see that too, but holds one more scalar register: 0.5 to 1 % of the large products.)
__device__ __forceinline__ void set_m0(uint32_t lds_addr) {
    uint32_t m0;
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0" : "={m0}"(m0) : "s"(lds_addr) : "memory");
}
template <int OFFSET>
__device__ __forceinline__ void dma16_at(int4v rsrc, uint32_t voff, uint32_t soff) {
    asm volatile("buffer_load_dwordx4 %0, %1, %2 offen offset:%3 lds" ::"v"(voff), "s"(rsrc), "s"(soff), "n"(OFFSET)
                 : "memory");
}

template <int I> using Int = std::integral_constant<int, I>;

// All but the N newest vector-memory operations of this wave are done, and every wave is here.
template <int N>
__device__ __forceinline__ void wait_and_barrier() {
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

}  // namespace nvfp4
