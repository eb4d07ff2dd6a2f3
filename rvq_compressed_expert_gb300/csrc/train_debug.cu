// The test aid of waste_train.h: a wait that gives up.
#include "train.cuh"

namespace wm {
namespace train {

namespace {
// The barrier is the CTA's own, and nobody arrives at it but thread 0, if asked to: the wait ends after so many polls.
__global__ void __launch_bounds__(32) debug_wait_kernel(uint32_t *word, bool rows, int polls, int arrive) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ uint32_t gave_up;
    const uint32_t at = tc::smem_u32(&bar);
    if (threadIdx.x == 0) {
        gave_up = 0;
        tc::mbar_init(at, 1);
        tc::mbar_init_fence();
        if (arrive) tc::mbar_arrive(at);
    }
    __syncwarp();
    if (rows) {
        for (int i = 0; i < 3; ++i) wait_row(at, 0, &gave_up, word, polls);
        settle(&gave_up);
    } else if (!tc::mbar_wait(at, 0, polls) && threadIdx.x == 0) {
        atomicOr(word, 1u);
    }
}
} // namespace

cudaError_t launch_debug_wait(uint32_t *word, bool rows, int polls, int arrive, cudaStream_t s) {
    debug_wait_kernel<<<1, 32, 0, s>>>(word, rows, polls, arrive);
    return cudaGetLastError();
}

} // namespace train
} // namespace wm
