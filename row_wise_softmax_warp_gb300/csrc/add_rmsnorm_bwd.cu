// add_rmsnorm_bwd.cu - the gradients of add_rmsnorm.cu.
//
//   n = h / rms,  g = dy * gamma,  t = dh + (g - n * mean_j(g_j n_j)) / rms
//   dresidual = t,  dx = drop(t),  dgamma_j = sum_i dy_ij n_ij
//
// dh is the gradient that arrives at h by the residual stream.  drop is the forward
// pass's mask, made again.  Bound by HBM: dy, h and dh are read once, dresidual and dx
// written once (16384 x 4096, bf16 and an fp32 stream, with dropout: 170 us, 6.3 TB/s; all
// bf16: 103 us, 5.2 TB/s); a warp takes 271 instructions for a row's 256 columns with dropout.
//
// A row lies in the registers of a group of lanes, of up to 16 warps, or of a cluster's CTAs
// (SPREAD below), which walk over rows and keep their columns' part of dgamma in registers;
// a block adds its sets of warps up in order and writes one row of partial sums, and a
// second launch adds those, all in an order that only the sizes, the alignment and the
// device decide.
#include <atomic>

#include "eight.cuh"
#include "pipeline.cuh"

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
    bool wide;  // long rows off 16-byte boundaries: the sums fit in shared memory
    int spread, span;  // CTAs of a cluster that share a row, and columns of each
};

// g and n of eight columns; adds to their products and to dgamma.
template <typename T, typename R, int LANES, bool VEC>
__device__ __forceinline__ void factors(const Held<T, LANES, VEC>& dy, const Held<R, LANES, VEC>& h, const float2 (&gamma)[4],
                                        float inv, float2 (&gy)[4], float2 (&n)[4], float2& dot, float2 (&dgamma)[4]) {
    dy.get(gy);
    h.get(n);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        n[i] = mul2(n[i], both(inv));
        dgamma[i] = fma2(gy[i], n[i], dgamma[i]);
        gy[i] = mul2(gy[i], gamma[i]);
        dot = fma2(gy[i], n[i], dot);
    }
}

template <typename T, typename R, int LANES, bool VEC>
__device__ __forceinline__ void gradients(const AddNormBwdArgs& a, const Masker& m, const Place<LANES, VEC>& o, int64_t row,
                                          int base, int g, const Held<R, LANES, VEC>& dh, const float2 (&gy)[4],
                                          const float2 (&n)[4], float inv, float mean) {
    float2 t[4], r[4];
    if (a.dh) dh.get(r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t[i] = mul2(fma2(n[i], both(-mean), gy[i]), both(inv));
        if (a.dh) t[i] = add2(t[i], r[i]);
    }
    if (a.dresidual) store_eight<LANES, VEC>(static_cast<R*>(a.dresidual), o, t);
    if (a.dx) {
        drop_eight<LANES, VEC>(t, a.drop, m, row, (a.cols + 7) / 8, base, g);
        store_eight<LANES, VEC>(static_cast<T*>(a.dx), o, t);
    }
}

// VEC: rows come through shared memory, where each thread keeps places for kStages rows of
// its own columns, so that the next rows are on their way while it works on one.  512 threads
// an SM then do (16384 x 4096, bf16 and fp32 stream with dropout: 170 us; 1024, which have
// half the registers, 177; without the places 181; three and four stages are no faster),
// in two blocks where a row takes 8 warps at most (4096 x 768 fp32: 13.6 us, in one 14.3).
// Rows that are read directly hide more behind 1024 threads (16384 x 1023: 67 us, 512: 77),
// whose 64 registers do not hold what a thread keeps: 48 to 56 bytes of it are spilled with one
// chunk a lane, 264 to 288 with two (rows of 4097 to 8192), in every row.
constexpr int kStages = 2;
template <typename T, typename R>
constexpr int kPlaces = Held<T, 32, true>::kChunks + 2 * Held<R, 32, true>::kChunks;  // of 16 bytes, a row

// SPREAD: the CTAs of a cluster share a row.  Each warp writes its part of the row's sum to
// every CTA, whose barrier counts the bytes (arrivals with a release would wait for the
// results' stores, row after row), and every warp, whose wait acquires at the cluster's scope
// as other CTAs wrote the parts, adds all of them in the same order.  A CTA is at most a row
// ahead of another: what it writes two rows later was read by then.
// Against one block a row, which reads dy and h twice: 4096 x 16384 bf16 121 and 184 us, 2048 x
// 32768 with an fp32 stream 173 and 273, 4096 x 10000 110 and 194, 3 x 12064 fp32 6.1 and 15.7.
constexpr int kMostSpread = 8;
template <bool SPREAD>
struct SpreadSums {
    float sums[2][kMostSpread * 16];
    uint64_t bar[2];
    int abort;
};
template <>
struct SpreadSums<false> {};

__device__ __forceinline__ void spread_part(float v, float* at, uint64_t* bar, uint32_t rank) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];\n" ::"r"(map_to_rank(at, rank)),
                 "f"(v), "r"(map_to_rank(bar, rank))
                 : "memory");
}

template <typename T, typename R, int LANES, int NV, bool VEC, int THREADS, bool SPREAD = false>
__global__ void __launch_bounds__(THREADS, VEC ? 512 / THREADS : 2) add_rmsnorm_bwd_rows(const AddNormBwdArgs a) {
    extern __shared__ __align__(16) float shared[];  // the places; afterwards sums of a.split.warps * NV * 256 columns
    __shared__ float scratch[2][32];
    __shared__ SpreadSums<SPREAD> all;
    let_next_start();
    // this CTA's columns, and its row among the clusters'
    int begin_col = 0, end_col = a.cols, group = blockIdx.x, groups = gridDim.x;
    if constexpr (SPREAD) {
        begin_col = int(cluster_rank()) * a.span;
        end_col = min(a.cols, begin_col + a.span);
        group = blockIdx.x / a.spread;
        groups = gridDim.x / a.spread;
        if (threadIdx.x == 0) {
            mbar_init(&all.bar[0], 1);
            mbar_init(&all.bar[1], 1);
            all.abort = 0;
            asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        }
        cluster_sync_all();  // with a release: this CTA's warps read the flag too
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot = warp / a.split.warps, w = warp % a.split.warps, g = lane % LANES;
    constexpr int kGroups = 32 / LANES;
    const float inv_cols = 1.0f / float(a.cols);
    const Masker masker(a.drop);
    const auto base_of = [&](int k) { return begin_col + (k * a.split.warps + w) * 256; };
    float2 gamma[NV][4], dgamma[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        load_weights<LANES, VEC>(a.gamma, Place<LANES, VEC>(0, 0, base_of(k), g, end_col), gamma[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) dgamma[k][i] = both(0.f);
    }

    using HeldT = Held<T, LANES, VEC>;
    using HeldR = Held<R, LANES, VEC>;
    const uint32_t step = blockDim.x * 16;  // from place to place
    const uint32_t places = uint32_t(__cvta_generic_to_shared(shared)) + threadIdx.x * 16;
    const int64_t first = (int64_t(group) * a.split.slots + slot) * kGroups;
    const int64_t stride = int64_t(groups) * a.split.slots * kGroups;
    const auto begin = [&](int64_t from, uint32_t at) {  // copies of the rows at `from`
        if constexpr (VEC) {
            const int64_t row = from + lane / LANES;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const Place<LANES, VEC> o(row, a.cols, base_of(k), g, row < a.rows ? end_col : 0);
                HeldT::copy(at, step, static_cast<const T*>(a.dy), o);
                at += HeldT::kChunks * step;
                HeldR::copy(at, step, static_cast<const R*>(a.h), o);
                at += HeldR::kChunks * step;
                if (a.dh) HeldR::copy(at, step, static_cast<const R*>(a.dh), o);
                at += HeldR::kChunks * step;
            }
            copies_end();
        }
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) begin(first + s * stride, places + s * NV * kPlaces<T, R> * step);
    const auto rms_at = [&](int64_t from) { return from + lane / LANES < a.rows ? __ldg(a.row_rms + from + lane / LANES) : 1.f; };
    float next_rms = VEC ? rms_at(first) : 0.f;  // asked for a row ahead
    int turn = 0;
    uint32_t phase = 0;
    for (int64_t from = first; from < a.rows; from += stride, turn ^= 1) {
        const int64_t row = from + lane / LANES;
        const int there = row < a.rows ? end_col : 0;
        const float inv = 1.0f / (VEC ? next_rms : rms_at(from));
        if (VEC) next_rms = rms_at(from + stride);
        HeldR dh[NV];
        float2 gy[NV][4], n[NV][4], dots = both(0.f);
        const uint32_t stage = places + turn * NV * kPlaces<T, R> * step;  // kStages is 2
        if constexpr (VEC) copies_wait<kStages - 1>();
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const Place<LANES, VEC> o(row, a.cols, base_of(k), g, there);
            const uint32_t at = stage + k * kPlaces<T, R> * step;
            HeldT dy;
            HeldR h;
            if constexpr (VEC) {
                dy.take(at, step, o);
                h.take(at + HeldT::kChunks * step, step, o);
            } else {
                dy.load(static_cast<const T*>(a.dy), o);
                h.load(static_cast<const R*>(a.h), o);
                if (a.dh) dh[k].load(static_cast<const R*>(a.dh), o);
            }
            factors<T, R, LANES, VEC>(dy, h, gamma[k], inv, gy[k], n[k], dots, dgamma[k]);
        }
        float dot;
        if constexpr (SPREAD) {
            const int parts = a.spread * a.split.warps;
            if (threadIdx.x == 0) mbar_arrive_expect_tx(&all.bar[turn], parts * 4);
            const float part = group_sum<32>(dots.x + dots.y);
            if (lane < a.spread) spread_part(part, &all.sums[turn][cluster_rank() * a.split.warps + w], &all.bar[turn], lane);
            if (!__all_sync(kFullMask, mbar_wait_cluster(&all.bar[turn], phase, &all.abort))) {
                if (lane == 0) raise_abort(&all.abort);
                break;
            }
            phase ^= turn;
            dot = 0.f;
            for (int i = lane; i < parts; i += 32) dot += all.sums[turn][i];
            dot = group_sum<32>(dot);
        } else {
            dot = sum_of_row<LANES>(dots.x + dots.y, scratch[turn], a.split.warps, slot, w);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const Place<LANES, VEC> o(row, a.cols, base_of(k), g, there);
            if constexpr (VEC) {
                if (a.dh) dh[k].take(stage + (k * kPlaces<T, R> + HeldT::kChunks + HeldR::kChunks) * step, step, o);
            }
            gradients<T, R, LANES, VEC>(a, masker, o, row, base_of(k), g, dh[k], gy[k], n[k], inv, dot * inv_cols);
        }
        begin(from + kStages * stride, stage);  // where all has been read
    }
    if constexpr (VEC) copies_wait<0>();
    __syncthreads();
    // the groups of a warp, then the sets of warps in order
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dgamma[k][i] = make_float2(across_groups_sum<LANES>(dgamma[k][i].x), across_groups_sum<LANES>(dgamma[k][i].y));
    for (int s = 0; s < a.split.slots; ++s) {
        if (slot == s && lane < LANES) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float* to = shared + base_of(k) - begin_col + (VEC ? 8 * g + i : i * LANES + g);
                    const float d = i & 1 ? dgamma[k][i / 2].y : dgamma[k][i / 2].x;
                    *to = s == 0 ? d : *to + d;
                }
        }
        __syncthreads();
    }
    for (int c = begin_col + threadIdx.x; c < end_col; c += blockDim.x) a.parts[int64_t(group) * a.cols + c] = shared[c - begin_col];
    if constexpr (SPREAD) {  // after a wait that was given up the others may still write here
        cluster_arrive_relaxed();
        cluster_wait();
    }
}

// dgamma = the blocks' parts, added in order within each warp and then over the warps: a
// warp 32 columns of every 32nd part.  A programmatic dependent of what writes them.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32) sum_parts(const float* parts, float* dgamma, int blocks, int cols) {
    __shared__ float sums[kSumWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    wait_for_earlier();
    float sum = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int b = warp; b < blocks; b += kSumWarps) sum += parts[int64_t(b) * cols + c];
    }
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < cols) {
#pragma unroll
        for (int q = 1; q < kSumWarps; ++q) sum += sums[q][lane];
        dgamma[c] = sum;
    }
}

// Rows of more than 65536 values, or of more than 8192 off 16-byte boundaries: one block a
// row.  dy and h are read a second time, from the L2.  The sums over rows lie in the block's
// row of parts, which is its own and stays in the L2, or, of rows off a boundary that fit
// (kWideCols), in shared memory.  A thread reads and writes its own columns only.
template <typename T, typename R, bool VEC>
__global__ void __launch_bounds__(1024) add_rmsnorm_bwd_long(const AddNormBwdArgs a) {
    extern __shared__ __align__(16) float sums[];
    __shared__ float scratch[2][32];
    let_next_start();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float inv_cols = 1.0f / float(a.cols);
    const Masker masker(a.drop);
    const int64_t units = (int64_t(a.cols) + 255) / 256;
    float* parts = a.parts + int64_t(blockIdx.x) * a.cols;
    const bool wide = !VEC && a.wide;
    float* mine = wide ? sums : parts;
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
        const float inv = 1.0f / __ldg(a.row_rms + row);
        const auto read = [&](int base, Held<T, 32, VEC>& dy, Held<R, 32, VEC>& h, float2 (&gamma)[4]) {
            const Place<32, VEC> o(row, a.cols, base, lane, a.cols);
            dy.load(static_cast<const T*>(a.dy), o);
            h.load(static_cast<const R*>(a.h), o);
            load_weights<32, VEC>(a.gamma, Place<32, VEC>(0, 0, base, lane, a.cols), gamma);
            return o;
        };
        float2 dots = both(0.f);
#pragma unroll VEC ? 2 : 1
        for (int64_t u = w; u < units; u += 32) {
            Held<T, 32, VEC> dy;
            Held<R, 32, VEC> h;
            float2 gamma[4], gy[4], n[4], none[4] = {};
            read(int(u * 256), dy, h, gamma);
            factors<T, R, 32, VEC>(dy, h, gamma, inv, gy, n, dots, none);
        }
        const float mean = sum_of_row<32>(dots.x + dots.y, scratch[turn], 32, 0, w) * inv_cols;
#pragma unroll VEC ? 2 : 1
        for (int64_t u = w; u < units; u += 32) {
            const int base = int(u * 256);
            Held<T, 32, VEC> dy;
            Held<R, 32, VEC> h, dh;
            float2 gamma[4], gy[4], n[4], none = both(0.f), dgamma[4] = {};
            const Place<32, VEC> o = read(base, dy, h, gamma);
            if (a.dh) dh.load(static_cast<const R*>(a.dh), o);
            factors<T, R, 32, VEC>(dy, h, gamma, inv, gy, n, none, dgamma);
            if constexpr (VEC) {
                if (o.left > 0) {
                    float4* sum = reinterpret_cast<float4*>(mine + base + 8 * lane);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float4 v = sum[q];
                        v.x += dgamma[2 * q].x, v.y += dgamma[2 * q].y, v.z += dgamma[2 * q + 1].x, v.w += dgamma[2 * q + 1].y;
                        sum[q] = v;
                    }
                }
            } else {
                each(base, [&](int col, int i) { mine[col] += i & 1 ? dgamma[i / 2].y : dgamma[i / 2].x; });
            }
            gradients<T, R, 32, VEC>(a, masker, o, row, base, lane, dh, gy, n, inv, mean);
        }
    }
    if (!wide) return;
    for (int64_t u = w; u < units; u += 32) each(int(u * 256), [&](int c, int) { parts[c] = sums[c]; });
}

constexpr int64_t kRegisterCols = 8192;  // 256 or 512 columns for each of the most warps of a row
constexpr int64_t kWideCols = 48 * 1024;  // sums in shared memory, of long rows off 16-byte boundaries

// Lanes, columns of a lane, warps and sets of warps by the row's length, and blocks by the
// rows.
struct BwdPlan {
    int lanes, nv, warps, slots;
    int threads;  // at most
    int64_t blocks;  // that write a row of parts: blocks, or clusters of `spread`
    int spread = 1, span = 0;
};
BwdPlan plan_of(int64_t rows, int64_t cols, bool vec) {
    const int64_t sms = sm_count() > 0 ? sm_count() : 132;
    if (vec && cols > kRegisterCols && cols <= kMostSpread * kRegisterCols) {
        BwdPlan p{32, 2, 0, 1, 512, 0, 2, 0};
        // more CTAs a row where there are rows for few (3 x 12064 fp32: by two 8.2 us, by eight 6.1)
        while (p.spread * kRegisterCols < cols || (p.spread < kMostSpread && rows * p.spread * 2 <= sms)) p.spread *= 2;
        p.span = int((cols + 256 * p.spread - 1) / (256 * p.spread)) * 256;
        p.warps = (p.span / 256 + 1) / 2;
        p.blocks = rows < sms / p.spread ? rows : sms / p.spread;
        return p;
    }
    if (cols > kRegisterCols) return {32, 1, 32, 1, 1024, rows < sms ? rows : sms};
    BwdPlan p;
    const int units = int((cols + 255) / 256);
    p.lanes = cols <= 64 ? 8 : cols <= 128 ? 16 : 32;
    p.nv = units > 16 ? 2 : 1;
    p.warps = (units + p.nv - 1) / p.nv;
    const bool half = vec && p.warps <= 8;  // of the block, twice
    p.threads = half ? 256 : 512;
    p.slots = p.threads / 32 / p.warps;
    const int64_t sets = (rows + p.slots - 1) / p.slots;
    const int64_t most = half || !vec ? 2 * sms : sms;
    p.blocks = sets < most ? sets : most;
    return p;
}

// Clusters of a.spread CTAs that the device runs at once (0 if unknown): one more than
// those would run behind them, as a second round.
template <auto kernel>
int64_t resident_clusters(cudaLaunchConfig_t cfg, int spread) {
    static std::atomic<int> cached[64][kMostSpread + 1];
    int dev = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev < 64)
        if (const int c = cached[dev][spread].load(std::memory_order_relaxed)) return c;
    cfg.blockDim = dim3(512);  // the most that any call takes
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();  // or it would be taken for the launch's
        return 0;
    }
    if (dev < 64) cached[dev][spread].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace

uint32_t pipeline_timeouts_norm() { return read_pipeline_timeouts(); }

size_t add_rmsnorm_bwd_workspace(int64_t rows, int64_t cols) {
    if (rows <= 0) return 0;  // of rows on 16-byte boundaries and others, whichever take more
    const int64_t a = plan_of(rows, cols, true).blocks, b = plan_of(rows, cols, false).blocks;
    return size_t(a > b ? a : b) * size_t(cols) * 4;
}

cudaError_t launch_add_rmsnorm_bwd(const void* dy, const float* gamma, const void* h, const float* row_rms,
                                   const void* dh, const uint64_t* rng, void* dresidual, void* dx, float* dgamma,
                                   int64_t rows, int64_t cols, float p, int x_type, int h_type, float* parts,
                                   cudaStream_t stream) {
    const bool vec = cols % 8 == 0 && ((reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(gamma) |
                                        reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(dh) |
                                        reinterpret_cast<uintptr_t>(dresidual) | reinterpret_cast<uintptr_t>(dx)) & 15) == 0;
    BwdPlan plan = plan_of(rows, cols, vec);
    // Without dx there is no mask to make, and rng may be NULL.
    AddNormBwdArgs a{dy,   gamma,     h,           row_rms, dh, dresidual, dx, parts, dropout_of(rng, dx ? p : 0.f),
                     rows, int(cols), {plan.warps, plan.slots}, cols <= kWideCols, plan.spread, plan.span};
    cudaError_t e = cudaSuccess;
    with_branch_types(x_type, h_type, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        auto go = [&](auto kernel, size_t smem) {
            if (smem > 32 * 1024) e = allow_smem(kernel, smem);  // 48 KB with the static part need no leave
            if (e == cudaSuccess) kernel<<<unsigned(plan.blocks), unsigned(plan.warps * plan.slots * 32), smem, stream>>>(a);
        };
        const size_t sums = size_t(plan.warps) * plan.nv * 256 * 4;
        const size_t staged = size_t(kStages) * plan.nv * kPlaces<T, R> * 16 * plan.warps * plan.slots * 32;
        const size_t smem = vec && staged > sums ? staged : sums;
        if (plan.spread > 1) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim = {unsigned(plan.spread), 1, 1};
            cfg.gridDim = dim3(unsigned(plan.spread));
            cfg.dynamicSmemBytes = size_t(kStages) * plan.nv * kPlaces<T, R> * 16 * 512;
            cfg.stream = stream;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            constexpr auto kernel = add_rmsnorm_bwd_rows<T, R, 32, 2, true, 512, true>;
            e = allow_smem(kernel, cfg.dynamicSmemBytes);
            if (e != cudaSuccess) return;
            const int64_t most = resident_clusters<kernel>(cfg, plan.spread);
            if (most > 0 && most < plan.blocks) plan.blocks = most;
            cfg.gridDim = dim3(unsigned(plan.blocks * plan.spread));
            cfg.blockDim = dim3(unsigned(plan.warps * 32));
            cfg.dynamicSmemBytes = smem;
            e = cudaLaunchKernelEx(&cfg, kernel, a);
        } else if (cols > kRegisterCols) {
            if (vec) go(add_rmsnorm_bwd_long<T, R, true>, 0);
            else go(add_rmsnorm_bwd_long<T, R, false>, a.wide ? size_t(cols) * 4 : 0);
        } else if (!vec) {
            if (plan.nv == 1) go(add_rmsnorm_bwd_rows<T, R, 32, 1, false, 512>, smem);
            else go(add_rmsnorm_bwd_rows<T, R, 32, 2, false, 512>, smem);
        } else if (plan.lanes == 8) go(add_rmsnorm_bwd_rows<T, R, 8, 1, true, 256>, smem);
        else if (plan.lanes == 16) go(add_rmsnorm_bwd_rows<T, R, 16, 1, true, 256>, smem);
        else if (plan.threads == 256) go(add_rmsnorm_bwd_rows<T, R, 32, 1, true, 256>, smem);
        else if (plan.nv == 1) go(add_rmsnorm_bwd_rows<T, R, 32, 1, true, 512>, smem);
        else go(add_rmsnorm_bwd_rows<T, R, 32, 2, true, 512>, smem);
    });
    if (e != cudaSuccess) return e;
    note_launches(2);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(unsigned((cols + 31) / 32));
    cfg.blockDim = dim3(kSumWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sum_parts, static_cast<const float*>(parts), dgamma, int(plan.blocks), int(cols));
}

}  // namespace rowops
