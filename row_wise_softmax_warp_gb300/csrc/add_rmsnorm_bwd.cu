// add_rmsnorm_bwd.cu - the gradients of add_rmsnorm.cu.
//
//   n = h / rms,  g = dy * gamma,  t = dh + (g - n * mean_j(g_j n_j)) / rms
//   dresidual = t,  dx = drop(t),  dgamma_j = sum_i dy_ij n_ij
//
// dh is the gradient that arrives at h by the residual stream.  drop is the forward
// pass's mask, made again.  Bound by HBM: dy, h and dh are read once, dresidual and dx
// written once.
//
// A row lies in the registers of a group of lanes or of up to 32 warps, which walk over
// rows and keep their columns' part of dgamma in registers; a block adds its sets of
// warps up in order and writes one row of partial sums, and column sums (rmsnorm.cu)
// add those, all in an order that only the sizes and the device decide.
#include "eight.cuh"

namespace rowops {
namespace {

struct AddNormBwdArgs {
    const void* dy;
    const float* gamma;
    const void* h;
    const float* row_rms;
    const void* dh;  // may be NULL
    void* dresidual;  // may be NULL
    void* dx;         // may be NULL
    float* parts;     // a row of cols for each block
    Dropout drop;
    int64_t rows;
    int cols;
    RowSplit split;
    bool wide;  // long rows: the sums fit in shared memory
};

template <typename T, typename R, int LANES, bool VEC>
__device__ __forceinline__ void gradients(const AddNormBwdArgs& a, const Masker& m, int64_t row, int base, int g,
                                          int cols, const Held<R, LANES, VEC>& dh, const float (&gy)[8],
                                          const float (&n)[8], float inv, float mean) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t[i] = (gy[i] - n[i] * mean) * inv;
        if (a.dh) t[i] += dh.get(i);
    }
    if (a.dresidual) store_eight<LANES, VEC>(static_cast<R*>(a.dresidual) + row * a.cols, base, g, cols, t);
    if (a.dx) {
        drop_eight<LANES, VEC>(t, a.drop, m, row, (a.cols + 7) / 8, base, g);
        store_eight<LANES, VEC>(static_cast<T*>(a.dx) + row * a.cols, base, g, cols, t);
    }
}

template <typename T, typename R, int LANES, bool VEC>
__global__ void __launch_bounds__(1024) add_rmsnorm_bwd_rows(const AddNormBwdArgs a) {
    extern __shared__ float sums[];  // a.split.warps * 256
    __shared__ float scratch[2][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot = warp / a.split.warps, w = warp % a.split.warps, g = lane % LANES;
    constexpr int kGroups = 32 / LANES;
    const float inv_cols = 1.0f / float(a.cols);
    const Masker masker(a.drop);
    const int base = w * 256;
    float gamma[8], dgamma[8];
    load_weights<LANES, VEC>(a.gamma, base, g, a.cols, gamma);
#pragma unroll
    for (int i = 0; i < 8; ++i) dgamma[i] = 0.f;
    int turn = 0;
    for (int64_t first = (int64_t(blockIdx.x) * a.split.slots + slot) * kGroups; first < a.rows;
         first += int64_t(gridDim.x) * a.split.slots * kGroups, turn ^= 1) {
        const bool live = first + lane / LANES < a.rows;
        const int64_t row = live ? first + lane / LANES : 0;
        const int cols = live ? a.cols : 0;
        Held<T, LANES, VEC> dy;
        Held<R, LANES, VEC> h, dh;
        dy.load(static_cast<const T*>(a.dy) + row * a.cols, base, g, cols);
        h.load(static_cast<const R*>(a.h) + row * a.cols, base, g, cols);
        if (a.dh) dh.load(static_cast<const R*>(a.dh) + row * a.cols, base, g, cols);
        const float inv = live ? 1.0f / __ldg(a.row_rms + row) : 0.f;
        float gy[8], n[8], dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = dy.get(i);
            n[i] = h.get(i) * inv;
            dgamma[i] = fmaf(d, n[i], dgamma[i]);
            gy[i] = d * gamma[i];
            dot = fmaf(gy[i], n[i], dot);
        }
        dot = sum_of_row<LANES>(dot, scratch[turn], a.split.warps, slot, w);
        gradients<T, R, LANES, VEC>(a, masker, row, base, g, cols, dh, gy, n, inv, dot * inv_cols);
    }
    // the groups of a warp, then the sets of warps in order
#pragma unroll
    for (int i = 0; i < 8; ++i) dgamma[i] = across_groups_sum<LANES>(dgamma[i]);
    for (int s = 0; s < a.split.slots; ++s) {
        if (slot == s && lane < LANES) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float* to = sums + base + (VEC ? 8 * g + i : i * LANES + g);
                *to = s == 0 ? dgamma[i] : *to + dgamma[i];
            }
        }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) a.parts[int64_t(blockIdx.x) * a.cols + c] = sums[c];
}

// Rows of more than 8192 values: one block a row.  dy and h are read a second time,
// from the L2, and the sums over rows lie in shared memory, or where that is too small in
// the block's row of parts.  A thread reads and writes its own columns only.
template <typename T, typename R, bool VEC>
__global__ void __launch_bounds__(1024) add_rmsnorm_bwd_long(const AddNormBwdArgs a) {
    extern __shared__ float sums[];
    __shared__ float scratch[2][32];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float inv_cols = 1.0f / float(a.cols);
    const Masker masker(a.drop);
    const int64_t units = (int64_t(a.cols) + 255) / 256;
    float* parts = a.parts + int64_t(blockIdx.x) * a.cols;
    float* mine = a.wide ? sums : parts;
    const auto each = [&](int base, auto&& f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = base + (VEC ? 8 * lane + i : i * 32 + lane);
            if (c < a.cols) f(c, i);
        }
    };
    for (int64_t u = w; u < units; u += 32) each(int(u * 256), [&](int c, int) { mine[c] = 0.f; });
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const T* dy_row = static_cast<const T*>(a.dy) + row * a.cols;
        const R* h_row = static_cast<const R*>(a.h) + row * a.cols;
        const float inv = 1.0f / __ldg(a.row_rms + row);
        float dot = 0.f;
        for (int64_t u = w; u < units; u += 32) {
            Held<T, 32, VEC> dy;
            Held<R, 32, VEC> h;
            float gamma[8];
            dy.load(dy_row, int(u * 256), lane, a.cols);
            h.load(h_row, int(u * 256), lane, a.cols);
            load_weights<32, VEC>(a.gamma, int(u * 256), lane, a.cols, gamma);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot = fmaf(dy.get(i) * gamma[i], h.get(i) * inv, dot);
        }
        dot = sum_of_row<32>(dot, scratch[turn], 32, 0, w);
        for (int64_t u = w; u < units; u += 32) {
            const int base = int(u * 256);
            Held<T, 32, VEC> dy;
            Held<R, 32, VEC> h, dh;
            float gy[8], n[8];
            dy.load(dy_row, base, lane, a.cols);
            h.load(h_row, base, lane, a.cols);
            if (a.dh) dh.load(static_cast<const R*>(a.dh) + row * a.cols, base, lane, a.cols);
            load_weights<32, VEC>(a.gamma, base, lane, a.cols, gy);
            each(base, [&](int col, int i) { mine[col] = fmaf(dy.get(i), h.get(i) * inv, mine[col]); });
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                n[i] = h.get(i) * inv;
                gy[i] *= dy.get(i);
            }
            gradients<T, R, 32, VEC>(a, masker, row, base, lane, a.cols, dh, gy, n, inv, dot * inv_cols);
        }
    }
    if (!a.wide) return;
    for (int64_t u = w; u < units; u += 32) each(int(u * 256), [&](int c, int) { parts[c] = sums[c]; });
}

constexpr int64_t kRegisterCols = 8192;  // one group of 256 columns for each of 32 warps
constexpr int64_t kWideCols = 48 * 1024;  // sums in shared memory

// Lanes, warps and sets of warps by the row's length, and blocks by the rows.
struct BwdPlan {
    int lanes, warps, slots;
    int64_t blocks;
};
BwdPlan plan_of(int64_t rows, int64_t cols) {
    const int64_t sms = sm_count() > 0 ? sm_count() : 132;
    if (cols > kRegisterCols) return {32, 32, 1, rows < sms ? rows : sms};
    BwdPlan p;
    const int units = int((cols + 255) / 256);
    p.lanes = cols <= 64 ? 8 : cols <= 128 ? 16 : 32;
    p.warps = units;
    p.slots = units >= 16 ? 1 : units >= 2 ? 16 / units : 8;
    const int64_t sets = (rows + p.slots - 1) / p.slots;
    p.blocks = sets < 2 * sms ? sets : 2 * sms;
    return p;
}

}  // namespace

size_t add_rmsnorm_bwd_workspace(int64_t rows, int64_t cols) {
    return rows > 0 ? size_t(plan_of(rows, cols).blocks) * size_t(cols) * 4 : 0;
}

cudaError_t launch_add_rmsnorm_bwd(const void* dy, const float* gamma, const void* h, const float* row_rms,
                                   const void* dh, const uint64_t* rng, void* dresidual, void* dx, float* dgamma,
                                   int64_t rows, int64_t cols, float p, int x_type, int h_type, float* parts,
                                   cudaStream_t stream) {
    const BwdPlan plan = plan_of(rows, cols);
    AddNormBwdArgs a{dy,   gamma,     h,           row_rms, dh, dresidual, dx, parts, dropout_of(rng, p),
                     rows, int(cols), {plan.warps, plan.slots}, cols <= kWideCols};
    const bool vec = cols % 8 == 0 && ((reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(gamma) |
                                        reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(dh) |
                                        reinterpret_cast<uintptr_t>(dresidual) | reinterpret_cast<uintptr_t>(dx)) & 15) == 0;
    cudaError_t e = cudaSuccess;
    auto go = [&](auto kernel, size_t smem) {
        if (smem > 32 * 1024) e = allow_smem(kernel, smem);  // 48 KB with the static part need no leave
        if (e != cudaSuccess) return;
        kernel<<<unsigned(plan.blocks), unsigned(plan.warps * plan.slots * 32), smem, stream>>>(a);
        note_launches(1);
        e = cudaGetLastError();
    };
    with_branch_types(x_type, h_type, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        const size_t smem = size_t(plan.warps) * 256 * 4;
        if (cols > kRegisterCols) {
            const size_t wide = a.wide ? size_t(cols) * 4 : 0;
            if (vec) go(add_rmsnorm_bwd_long<T, R, true>, wide);
            else go(add_rmsnorm_bwd_long<T, R, false>, wide);
        } else if (!vec) go(add_rmsnorm_bwd_rows<T, R, 32, false>, smem);
        else if (plan.lanes == 8) go(add_rmsnorm_bwd_rows<T, R, 8, true>, smem);
        else if (plan.lanes == 16) go(add_rmsnorm_bwd_rows<T, R, 16, true>, smem);
        else go(add_rmsnorm_bwd_rows<T, R, 32, true>, smem);
    });
    if (e != cudaSuccess) return e;
    return launch_column_sums(parts, dgamma, plan.blocks, cols, 0.f, stream);
}

}  // namespace rowops
