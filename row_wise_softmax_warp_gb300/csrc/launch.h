// launch.h - host-side glue between the C ABI (abi.cu) and the kernels.
//
// Each launch_* function queues the kernel(s) of one op on `stream` for
// arguments that abi.cu has already validated, and returns the CUDA error of
// the launch.  `vec4` says that every row-major matrix argument is 16-byte
// aligned with cols % 4 == 0 (and byte masks 4-byte aligned), which enables the
// 128-bit path.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace rowops {

// ------------------------------------------------------------ bookkeeping

void note_launches(int n);  // counts kernels queued (rowops_kernel_launches)
int sm_count();             // SMs of the current device (cached; 0 if unknown)

// Allows launches of `kernel` on the current device `bytes` of dynamic shared memory.
// The limit belongs to the function on the device and not to a call, so it is only
// ever raised: a host thread that needs less must not lower it between another's
// call of this function and its launch.
cudaError_t allow_smem(const void* kernel, size_t bytes);
template <typename... A>
cudaError_t allow_smem(void (*kernel)(A...), size_t bytes) {
    return allow_smem(reinterpret_cast<const void*>(kernel), bytes);
}

template <int L, int N, int V>
struct Geom {
    static constexpr int LANES = L;
    static constexpr int NV = N;
    static constexpr int VEC = V;
};

// Calls f(Geom<LANES, NV, VEC>{}) with the group geometry for rows of `cols`
// floats (see common.cuh), or returns false when a row is longer than one
// warp holds in registers (1024 floats, vectorised or scalar).  Scalar rows
// keep the floats per lane of vectorised rows of the same length (NV = 32
// scalars against NV = 8 float4s); groups of at least 8 lanes make each row's
// share of a warp load one full 32-byte sector.
template <typename F>
bool with_geometry(bool vec4, int64_t cols, F&& f) {
    if (vec4) {
        const int64_t nc = cols / 4;
        if (nc <= 4) f(Geom<4, 1, 4>{});
        else if (nc <= 8) f(Geom<4, 2, 4>{});
        else if (nc <= 16) f(Geom<8, 2, 4>{});
        else if (nc <= 32) f(Geom<16, 2, 4>{});
        else if (nc <= 64) f(Geom<32, 2, 4>{});
        else if (nc <= 128) f(Geom<32, 4, 4>{});
        else if (nc <= 192) f(Geom<32, 6, 4>{});
        else if (nc <= 256) f(Geom<32, 8, 4>{});
        else return false;
    } else {
        if (cols <= 4) f(Geom<4, 1, 1>{});
        else if (cols <= 8) f(Geom<8, 1, 1>{});
        else if (cols <= 16) f(Geom<8, 2, 1>{});
        else if (cols <= 32) f(Geom<8, 4, 1>{});
        else if (cols <= 64) f(Geom<8, 8, 1>{});
        else if (cols <= 128) f(Geom<16, 8, 1>{});
        else if (cols <= 256) f(Geom<32, 8, 1>{});
        else if (cols <= 512) f(Geom<32, 16, 1>{});
        else if (cols <= 768) f(Geom<32, 24, 1>{});
        else if (cols <= 1024) f(Geom<32, 32, 1>{});
        else return false;
    }
    return true;
}

// Blocks of 256 threads for a group kernel over `rows` rows (grid-stride
// beyond the cap).
inline unsigned group_grid(int64_t rows, int lanes) {
    const int64_t groups_per_block = 256 / lanes;
    int64_t b = (rows + groups_per_block - 1) / groups_per_block;
    if (b > (1 << 20)) b = 1 << 20;
    return static_cast<unsigned>(b < 1 ? 1 : b);
}

// Balanced launch for a group kernel whose block is any whole number of warps
// (up to 1024 threads, GPB = blockDim.x / LANES): one block per SM holding
// ceil(rows / SMs) groups, so no SM carries a block more than another (with
// 256-thread blocks, 4096 rows of 768 floats put 4 blocks on 56 SMs and 3 on
// the other 96).  threads = 0 when that block would be smaller than
// kBlockThreads-equivalent work or larger than 1024 threads (use group_grid).
struct BalancedLaunch {
    unsigned grid = 0, threads = 0;
};
inline BalancedLaunch balanced_groups(int64_t rows, int lanes) {
    BalancedLaunch b;
    const int sms = sm_count();
    if (sms <= 0 || rows <= 0) return b;
    const int64_t per_sm = (rows + sms - 1) / sms;  // groups per block
    const int64_t nt = (per_sm * lanes + 31) / 32 * 32;
    if (nt < 256 || nt > 1024) return b;
    b.grid = static_cast<unsigned>((rows + per_sm - 1) / per_sm);
    b.threads = static_cast<unsigned>(nt);
    return b;
}

// Blocks for a group kernel whose loop loads the next rows while it works on
// the current ones: at most `per_sm` blocks per SM, so each group walks several
// rows and its loads stay in flight across the selection work.
inline unsigned stream_grid(int64_t rows, int lanes, int per_sm = 8) {
    const unsigned g = group_grid(rows, lanes);
    const int sms = sm_count();
    const int64_t cap = int64_t(sms > 0 ? sms : 132) * per_sm;
    return int64_t(g) > cap ? static_cast<unsigned>(cap) : g;
}

// Blocks for a one-row-per-block (or per-cluster) kernel.
inline unsigned row_grid(int64_t rows, int per_row = 1) {
    int64_t b = rows;
    const int64_t cap = (int64_t(1) << 20);
    if (b > cap) b = cap;
    return static_cast<unsigned>((b < 1 ? 1 : b) * per_row);
}

// ----------------------------------------------------------------- ops

cudaError_t launch_softmax_fwd(const float* x, float* y, int64_t rows, int64_t cols, bool vec4,
                               cudaStream_t stream);
// TMA-streamed long rows (tma_rows.cu): rows of more than 1024 floats from
// 4-byte aligned buffers (an output row must share its input row's alignment
// modulo 16 bytes); each returns false, launching nothing, when the shape does
// not suit it (the row does not fit in shared memory where it must stay
// resident, or the alignments differ).
bool launch_lse_tma(const float* x, float* lse, int64_t rows, int64_t cols, cudaStream_t stream,
                    cudaError_t* err);
bool launch_ce_tma(const float* x, const int32_t* targets, float* grad, float* row_loss, int64_t rows,
                   int64_t cols, float grad_scale, cudaStream_t stream, cudaError_t* err);
bool launch_softmax_tma(const float* x, float* y, int64_t rows, int64_t cols, cudaStream_t stream,
                        cudaError_t* err);
// Two-input long rows (weighted-logits and fixed-teacher CE): x and w must
// share their alignment modulo 16 bytes; grad (which may be NULL) may differ.
bool launch_soft_ce_tma(const float* x, const float* w, float* grad, float* row_loss, int64_t rows, int64_t cols,
                        float grad_scale, cudaStream_t stream, cudaError_t* err);
bool launch_teacher_ce_tma(const float* s, const float* t, float* grad, float* row_loss, int64_t rows,
                           int64_t cols, float grad_scale, cudaStream_t stream, cudaError_t* err);
// Timeouts counted by the bounded waits of each bulk-copy translation unit
// (rowops_pipeline_timeouts adds them up).
uint32_t pipeline_timeouts_rows();
uint32_t pipeline_timeouts_pairs();
uint32_t pipeline_timeouts_ln();
uint32_t pipeline_timeouts_matmul();
uint32_t pipeline_timeouts_fp8();
// LayerNorm backward stage 1 on rows of 384..1024 floats on 16-byte
// boundaries through the bulk-copy ring (one CTA per SM, at most 2^17 / cols
// and at most max_ctas, 0: no further limit); writes
// ln_bwd_tma_ctas(rows, cols, max_ctas) partials to ws.
// ln_bwd_tma_ctas is 0 for shapes it does not take.
int64_t ln_bwd_tma_ctas(int64_t rows, int64_t cols, int64_t max_ctas);
bool launch_ln_bwd_tma(const float* dy, const float* gamma, const float* xhat, const float* inv_std, float* dx,
                       float* ws, int64_t rows, int64_t cols, int64_t max_ctas, cudaStream_t stream,
                       cudaError_t* err);
// Softmax backward on long rows (two passes through the ring); y and dy must
// share their alignment modulo 16 bytes.
bool launch_softmax_bwd_tma(const float* y, const float* dy, float* dx, int64_t rows, int64_t cols,
                            cudaStream_t stream, cudaError_t* err);
cudaError_t launch_softmax_bwd(const float* y, const float* dy, float* dx, int64_t rows,
                               int64_t cols, bool vec4, cudaStream_t stream);
cudaError_t launch_attn_fwd(const float* s, float* p, int64_t rows, int64_t cols, int64_t seq_len,
                            float scale, bool vec4, cudaStream_t stream);
cudaError_t launch_attn_bwd(const float* p, const float* dp, float* ds, int64_t rows,
                            int64_t cols, int64_t seq_len, float scale, bool vec4,
                            cudaStream_t stream);
cudaError_t launch_masked_softmax(const float* x, const uint8_t* mask, float* y, int64_t rows,
                                  int64_t cols, bool vec4, cudaStream_t stream);
cudaError_t launch_logsumexp(const float* x, float* lse, int64_t rows, int64_t cols, bool vec4,
                             cudaStream_t stream);
cudaError_t launch_softmax_ce(const float* logits, const int32_t* targets, float* grad,
                              float* row_loss, double* mean_loss, int64_t rows, int64_t cols,
                              float grad_scale, bool vec4, cudaStream_t stream);
cudaError_t launch_layernorm_fwd(const float* x, const float* gamma, const float* beta,
                                 float* out, float* xhat, float* inv_std, int64_t rows,
                                 int64_t cols, float eps, bool vec4, cudaStream_t stream);
// The argument checks of rowops_layernorm_bwd other than the workspace's
// (dimensions, null and misaligned pointers, overlaps of the inputs and
// outputs), in the order that entry point reports them; sets *vec4.
int layernorm_bwd_checks(const float* dy, const float* gamma, const float* xhat, const float* inv_std, float* dx,
                         float* dgamma, float* dbeta, int64_t rows, int64_t cols, bool* vec4);
// budget (bytes, 0: none) caps the workspace the launch may use: the
// allocation-free entry point passes the size of its fixed array.
size_t layernorm_bwd_workspace(int64_t rows, int64_t cols, size_t budget = 0);
cudaError_t launch_layernorm_bwd(const float* dy, const float* gamma, const float* xhat,
                                 const float* inv_std, float* dx, float* dgamma, float* dbeta,
                                 int64_t rows, int64_t cols, float* workspace, bool vec4,
                                 cudaStream_t stream, size_t budget = 0);
cudaError_t launch_router(const float* x, const uint8_t* mask, float* p, float* kept, int64_t rows,
                          int64_t cols, int64_t k, bool vec4, cudaStream_t stream);
cudaError_t launch_top_k_rows(const float* x, float* values, float* indices, int64_t rows, int64_t cols,
                              int64_t k, bool largest, bool vec4, cudaStream_t stream);
cudaError_t launch_rmsnorm_fwd(const float* x, const float* gamma, float* out, float* row_rms, int64_t rows,
                               int64_t cols, float eps, bool vec4, cudaStream_t stream);
cudaError_t launch_rmsnorm_bwd(const float* dy, const float* gamma, const float* x, const float* row_rms,
                               float* dx, float* terms, int64_t rows, int64_t cols, bool vec4,
                               cudaStream_t stream);
cudaError_t launch_column_sums(const float* in, float* out, int64_t rows, int64_t cols, float beta,
                               cudaStream_t stream);
cudaError_t launch_masked_softmax_fmask(const float* x, const float* mask, float* y, int64_t rows,
                                        int64_t cols, bool vec4, cudaStream_t stream);
cudaError_t launch_lrp_softmax(const float* x, const float* y, const float* r, float* r_in, int64_t rows,
                               int64_t cols, bool vec4, cudaStream_t stream);
cudaError_t launch_argmax_onehot(const float* x, float* out, int64_t rows, int64_t cols, bool vec4,
                                 cudaStream_t stream);
// Fixed-order mean of the row losses into one double (programmatic dependent).
cudaError_t launch_row_mean(const float* row_loss, int64_t rows, double* mean_loss, cudaStream_t stream);
cudaError_t launch_soft_ce(const float* x, const float* w, float* grad, float* row_loss, double* mean_loss,
                           int64_t rows, int64_t cols, float grad_scale, bool vec4, cudaStream_t stream);
cudaError_t launch_teacher_ce(const float* s, const float* t, float* grad, float* row_loss, double* mean_loss,
                              int64_t rows, int64_t cols, float grad_scale, bool vec4, cudaStream_t stream);
cudaError_t launch_topk_kept(const float* x, float* kept, int64_t rows, int64_t cols, int64_t k,
                             bool vec4, cudaStream_t stream);

// The expert operators (types are rowops_dtype values).
size_t expert_plan_workspace(int64_t pairs, int64_t experts);
cudaError_t launch_expert_plan(const float* indices, const float* values, int32_t* offsets, int32_t* order,
                               int32_t* slot, int64_t pairs, int64_t experts, void* workspace, cudaStream_t stream);
cudaError_t launch_expert_gather(const void* x, const int32_t* slot, void* out, int64_t rows, int64_t k,
                                 int64_t cols, int64_t slots, int x_type, int out_type, cudaStream_t stream);
cudaError_t launch_expert_combine(const void* y, const int32_t* slot, const float* weights, void* out, int64_t rows,
                                  int64_t k, int64_t cols, int64_t slots, int y_type, int out_type,
                                  cudaStream_t stream);
cudaError_t launch_expert_combine_bwd(const void* dout, const void* y, const int32_t* slot, const float* weights,
                                      void* dy, float* dweights, int64_t rows, int64_t k, int64_t cols,
                                      int64_t slots, int out_type, int y_type, cudaStream_t stream);
cudaError_t launch_quantize_blocks(const void* x, uint8_t* q, float* scale, int64_t batches, int64_t rows,
                                   int64_t cols, int64_t block_rows, int x_type, cudaStream_t stream);
// Scratch memory of one call: `take` gives 256-byte aligned parts of it in turn.
struct Scratch {
    void* p;
    size_t bytes;
    void* take(size_t n) {
        n = (n + 255) & ~size_t(255);
        if (p == nullptr || n > bytes) return nullptr;
        void* part = p;
        p = static_cast<char*>(p) + n;
        bytes -= n;
        return part;
    }
};

// Rows copied to rows on 16-byte boundaries.  rows_per_expert > 0: rows of
// experts without a group in `offsets` may be left out.
struct RepackJob {
    const void* src;
    void* dst;
    int64_t rows, row_bytes, rows_per_expert;
};
__host__ __device__ inline int64_t repack_pitch(int64_t row_bytes) { return (row_bytes + 15) & ~int64_t(15); }
inline size_t repack_bytes(int64_t rows, int64_t row_bytes) { return size_t(rows * repack_pitch(row_bytes) + 255) & ~size_t(255); }
cudaError_t launch_repack(const RepackJob* jobs, int n, const int32_t* offsets, int64_t slots, cudaStream_t stream);

cudaError_t launch_expert_matmul(const void* x, const void* w, const int32_t* offsets, void* y, int64_t slots,
                                 int64_t in, int64_t out, int64_t experts, bool transposed, int dtype,
                                 Scratch scratch, cudaStream_t stream);
cudaError_t launch_expert_matmul_wgrad(const void* dy, const void* x, const int32_t* offsets, void* dw,
                                       int64_t slots, int64_t in, int64_t out, int64_t experts, int dtype,
                                       int dw_type, Scratch scratch, cudaStream_t stream);
cudaError_t launch_expert_matmul_fp8(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                                     const int32_t* offsets, void* y, int64_t slots, int64_t in, int64_t out,
                                     int64_t experts, int y_type, Scratch scratch, cudaStream_t stream);
// The same products for matrices of any alignment, without scratch memory.
cudaError_t launch_matmul_any(const void* x, const void* w, const int32_t* offsets, void* y, int64_t slots,
                              int64_t in, int64_t out, int64_t experts, bool transposed, int dtype,
                              cudaStream_t stream);
cudaError_t launch_matmul_wgrad_any(const void* dy, const void* x, const int32_t* offsets, void* dw, int64_t slots,
                                    int64_t in, int64_t out, int64_t experts, int dtype, int dw_type,
                                    cudaStream_t stream);
cudaError_t launch_matmul_fp8_any(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                                  const int32_t* offsets, void* y, int64_t slots, int64_t in, int64_t out,
                                  int64_t experts, int y_type, cudaStream_t stream);

}  // namespace rowops
