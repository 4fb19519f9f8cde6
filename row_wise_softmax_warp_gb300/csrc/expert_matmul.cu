// expert_matmul.cu - the experts' matrix products.
#include "launch.h"

namespace rowops {

cudaError_t launch_expert_matmul(const void* x, const void* w, const int32_t* offsets, void* y, int64_t slots,
                                 int64_t in, int64_t out, int64_t experts, bool transposed, int dtype,
                                 cudaStream_t stream) {
    return launch_matmul_any(x, w, offsets, y, slots, in, out, experts, transposed, dtype, stream);
}

cudaError_t launch_expert_matmul_wgrad(const void* dy, const void* x, const int32_t* offsets, void* dw,
                                       int64_t slots, int64_t in, int64_t out, int64_t experts, int dtype,
                                       int dw_type, cudaStream_t stream) {
    return launch_matmul_wgrad_any(dy, x, offsets, dw, slots, in, out, experts, dtype, dw_type, stream);
}

cudaError_t launch_expert_matmul_fp8(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                                     const int32_t* offsets, void* y, int64_t slots, int64_t in, int64_t out,
                                     int64_t experts, int y_type, cudaStream_t stream) {
    return launch_matmul_fp8_any(x, x_scale, w, w_scale, offsets, y, slots, in, out, experts, y_type, stream);
}

}  // namespace rowops
