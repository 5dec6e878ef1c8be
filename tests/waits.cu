// A kernel of one warp over the waits of csrc/barrier.cuh, with short limits, for tests/test_gpu_waits.py.
#include "barrier.cuh"

using namespace fathom;

namespace {

constexpr uint32_t kShort = 1u << 15;

// out: [0] gave up on a barrier that nothing arrives at, [1] waits again although it gave up,
// [2] gives up without time on a barrier that is complete, [3] gave up on a barrier that is complete
__global__ void waits_kernel(int wait_for_nothing, int* out, unsigned int* status) {
    __shared__ uint64_t empty, full;
    if (threadIdx.x == 0) {
        barrier_init(&empty, 1);
        barrier_init(&full, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    barrier_arrive(&full);
    __syncwarp();
    const bool late = barrier_gives_up<0>(&full, 0);
    bool fine = false, stuck = false;
    barrier_wait<kShort>(&full, 0, fine);
    bool again = false;
    if (wait_for_nothing) {
        barrier_wait<kShort>(&empty, 0, stuck);
        const uint32_t start = (uint32_t)clock();
        barrier_wait<0x7FFFFFFFu>(&empty, 0, stuck);
        again = (uint32_t)clock() - start > 0x3FFFFFFFu;
    }
    if (threadIdx.x == 0) out[0] = stuck, out[1] = again, out[2] = late, out[3] = fine;
    barrier_report<kShort>(stuck, status);
}

}  // namespace

extern "C" int waits_run(int wait_for_nothing, int* out, unsigned int* status) {
    waits_kernel<<<1, 32>>>(wait_for_nothing, out, status);
    return (int)cudaGetLastError();
}
