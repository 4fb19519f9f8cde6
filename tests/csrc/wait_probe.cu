// Test-only: the long wait of the expert products by itself.  Warp 0 waits with
// a budget of `polls` polls on a barrier; warp 1 counts up the progress `steps`
// times, `gap` clocks apart, and then arrives (arrive != 0) or just leaves.
#include "tensor_core.cuh"

using namespace rowops;

__global__ void wait_probe(uint32_t polls, int steps, long long gap, int arrive, int* out) {
    __shared__ uint64_t bar;
    __shared__ int abort_word;
    __shared__ uint32_t progress_word;
    volatile uint32_t* progress = &progress_word;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort_word = 0;
        progress_word = 0;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const bool ok = warp_wait_stages(&bar, 0, &abort_word, progress, polls);
        if (threadIdx.x == 0) out[0] = ok;
    } else {
        for (int i = 1; i <= steps; ++i) {
            const long long until = clock64() + gap;
            while (clock64() < until) {
            }
            if (threadIdx.x == 32) *progress = uint32_t(i);
        }
        if (arrive && threadIdx.x == 32) mbar_arrive(&bar);
    }
    __syncthreads();
    if (threadIdx.x == 0) out[1] = abort_word;
}

extern "C" int run_wait_probe(uint32_t polls, int steps, long long gap, int arrive, int* out) {
    wait_probe<<<1, 64>>>(polls, steps, gap, arrive, out);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? int(e) : int(cudaDeviceSynchronize());
}

extern "C" unsigned run_wait_probe_timeouts() { return read_pipeline_timeouts(); }
