// Barriers in shared memory that asynchronous copies arrive at, and waits on them that end in any case.
#pragma once

#include "fathom_internal.cuh"

namespace fathom {

// A wait gives up after this many clocks, about a second, which no correct run reaches.  The warp then waits
// no more and issues no further copy; before it leaves it gives the copies in flight as long once more.
constexpr uint32_t kWaitClocks = 1u << 31;

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void barrier_init(uint64_t* b, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ bool barrier_try(uint64_t* b, uint32_t parity) {
    uint32_t done;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(done)
                 : "r"(smem_addr(b)), "r"(parity)
                 : "memory");
    return done != 0;
}
// The last try comes after the limit: a warp that was kept from running past it finds what has arrived meanwhile.
template <uint32_t CLOCKS>
__device__ __noinline__ bool barrier_gives_up(uint64_t* b, uint32_t parity) {
    const uint32_t start = (uint32_t)clock();
    while ((uint32_t)clock() - start < CLOCKS)
        if (barrier_try(b, parity)) return false;
    return !barrier_try(b, parity);
}
template <uint32_t CLOCKS = kWaitClocks>
__device__ __forceinline__ void barrier_wait(uint64_t* b, uint32_t parity, bool& stuck) {
    if (!barrier_try(b, parity) && !stuck) stuck = barrier_gives_up<CLOCKS>(b, parity);
}
// the end of a warp's part, behind its last wait
template <uint32_t CLOCKS = kWaitClocks>
__device__ __forceinline__ void barrier_report(bool stuck, unsigned int* status) {
    if (!stuck) return;
    const uint32_t start = (uint32_t)clock();
    while ((uint32_t)clock() - start < CLOCKS) {}
    atomicOr(status, (unsigned)FATHOM_DEV_TIMEOUT);
}
// bytes to come before the barrier's phase is over
__device__ __forceinline__ void barrier_expect(uint64_t* b, uint32_t bytes) {
    asm volatile("{ .reg .b64 t; mbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1; }" ::"r"(smem_addr(b)), "r"(bytes) : "memory");
}
// this warp has read what the barrier's buffer held
__device__ __forceinline__ void barrier_arrive(uint64_t* b) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        asm volatile("{ .reg .b64 t; mbarrier.arrive.shared::cta.b64 t, [%0]; }" ::"r"(smem_addr(b)) : "memory");
}

}  // namespace fathom
