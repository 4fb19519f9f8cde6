// Test-only, included ahead of add_rmsnorm_bwd.cu: its calls of the CUDA runtime answered
// on the host.  The query of resident clusters fails as the runtime's does, which also
// leaves its error behind as the last one; launches are counted and succeed.
#pragma once
#include <cuda_runtime.h>

namespace fake {

inline cudaError_t last = cudaSuccess;
inline int launched = 0;
inline unsigned first_grid = 0;

inline cudaError_t get_device(int* dev) {
    *dev = 0;
    return cudaSuccess;
}
template <typename K>
cudaError_t max_active_clusters(int*, K, const cudaLaunchConfig_t*) {
    return last = cudaErrorInvalidClusterSize;
}
inline cudaError_t get_last_error() {
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
template <typename... P, typename... A>
cudaError_t launch(const cudaLaunchConfig_t* cfg, void (*)(P...), A&&...) {
    if (launched++ == 0) first_grid = cfg->gridDim.x;
    return cudaSuccess;
}

}  // namespace fake

#define cudaGetDevice fake::get_device
#define cudaOccupancyMaxActiveClusters fake::max_active_clusters
#define cudaGetLastError fake::get_last_error
#define cudaLaunchKernelEx fake::launch
