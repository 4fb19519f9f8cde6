// Test-only: launch_add_rmsnorm_bwd on rows that a cluster shares, where the query of
// resident clusters fails.  Nothing runs on a GPU.
#include "fake_cluster_query.h"

#include "add_rmsnorm_bwd.cu"

namespace rowops {
void note_launches(int) {}
int sm_count() { return 152; }
cudaError_t allow_smem(const void*, size_t) { return cudaSuccess; }
}  // namespace rowops

// out: the launcher's status, launches, the first one's blocks, the error left behind
extern "C" void run_cluster_query_probe(int* out) {
    const uintptr_t at = 1 << 20;
    void* p = reinterpret_cast<void*>(at);
    float* f = reinterpret_cast<float*>(at);
    out[0] = rowops::launch_add_rmsnorm_bwd(p, f, p, f, nullptr, nullptr, p, nullptr, f, 400, 16384, 0.f, 0, 0, f, nullptr);
    out[1] = fake::launched;
    out[2] = int(fake::first_grid);
    out[3] = fake::last;
}
