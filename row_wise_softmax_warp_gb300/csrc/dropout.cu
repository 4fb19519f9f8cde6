// dropout.cu - dropout from a counter-based generator, with a residual's addition.
//
//   y = residual + [u >= t] * x * 65536 / (65536 - t),   t = round(65536 p)
//
// u: 16 bits for each value (philox.cuh).  On a gradient, without a residual, the same
// call is the backward pass.  Bound by HBM where a value takes 6 bytes or more (98304 x
// 1024 fp32: 117 us, 6.9 TB/s; 16384 x 4096 bf16 with a residual: 61 us, 6.6 TB/s); of 4
// bytes a value the generator's instructions take part (16384 x 4096 bf16: 47 us, 5.8
// TB/s with four blocks a thread on their way, 53 with one).
#include "eight.cuh"

namespace rowops {
namespace {

constexpr int kDropThreads = 256;

struct DropoutArgs {
    const void* x;
    const void* residual;  // may be NULL
    void* y;
    Dropout drop;
    int64_t rows;
    int cols, units;  // units: groups of 8 * LANES columns in a row
    int64_t items;    // rows * units; of dropout_run: blocks of 8 of the matrix
};

// Rows that are whole blocks of 8 on 16-byte boundaries: the matrix as one run of them,
// ITEMS a thread, whose loads are on their way together.
template <typename T, typename R, int ITEMS>
__global__ void __launch_bounds__(kDropThreads) dropout_run(const DropoutArgs a) {
    const Masker masker(a.drop);
    const int64_t first = int64_t(blockIdx.x) * (kDropThreads * ITEMS) + threadIdx.x;
    const auto place = [&](int n) {
        const int64_t block = first + n * kDropThreads;
        return Place<32, true>(block, 8, 0, 0, block < a.items ? 8 : 0);
    };
    Held<T, 32, true> x[ITEMS];
    Held<R, 32, true> residual[ITEMS];
#pragma unroll
    for (int n = 0; n < ITEMS; ++n) {
        x[n].load(static_cast<const T*>(a.x), place(n));
        if (a.residual) residual[n].load(static_cast<const R*>(a.residual), place(n));
    }
#pragma unroll
    for (int n = 0; n < ITEMS; ++n) {
        float2 v[4];
        x[n].get(v);
        drop_eight<32, true>(v, a.drop, masker, first + n * kDropThreads, 1, 0, 0);
        if (a.residual) {
            float2 r[4];
            residual[n].get(r);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = add2(v[i], r[i]);
        }
        store_eight<32, true>(static_cast<R*>(a.y), place(n), v);
    }
}

// Other rows: a group of lanes takes 8 * LANES columns at a time.
template <typename T, typename R, int LANES>
__global__ void __launch_bounds__(kDropThreads) dropout_rows(const DropoutArgs a) {
    const int g = threadIdx.x % LANES;
    const Masker masker(a.drop);
    constexpr int kGroups = kDropThreads / LANES;
    const int64_t step = int64_t(gridDim.x) * kGroups;
    // A warp's groups stay together for the shuffles, so the loop goes by the warp's first.
    const int64_t first = int64_t(blockIdx.x) * kGroups + threadIdx.x / 32 * (32 / LANES);
    for (int64_t from = first; from < a.items; from += step) {
        const int64_t item = from + threadIdx.x % 32 / LANES, row = item / a.units;
        const int base = int(item - row * a.units) * 8 * LANES;
        const Place<LANES, false> o(row, a.cols, base, g, item < a.items ? a.cols : 0);
        Held<T, LANES, false> x;
        Held<R, LANES, false> residual;
        x.load(static_cast<const T*>(a.x), o);
        if (a.residual) residual.load(static_cast<const R*>(a.residual), o);
        float2 v[4];
        x.get(v);
        drop_eight<LANES, false>(v, a.drop, masker, row, (a.cols + 7) / 8, base, g);
        if (a.residual) {
            float2 r[4];
            residual.get(r);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = add2(v[i], r[i]);
        }
        store_eight<LANES, false>(static_cast<R*>(a.y), o, v);
    }
}

}  // namespace

cudaError_t launch_dropout(const void* x, const void* residual, const uint64_t* rng, void* y, int64_t rows,
                           int64_t cols, float p, int x_type, int y_type, cudaStream_t stream) {
    const bool vec = cols % 8 == 0 && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) |
                                        reinterpret_cast<uintptr_t>(y)) & 15) == 0;
    // Short rows share a warp (262144 x 33 bf16: 89 -> 25 us).
    const int lanes = cols <= 64 ? 8 : cols <= 128 ? 16 : 32;
    DropoutArgs a{x, residual, y, dropout_of(rng, p), rows, int(cols), int((cols + 8 * lanes - 1) / (8 * lanes)), 0};
    a.items = vec ? rows * (cols / 8) : rows * a.units;
    auto grid = [&](int64_t per) {
        const int64_t blocks = (a.items + per - 1) / per;
        return unsigned(vec || blocks < (1 << 20) ? blocks : 1 << 20);
    };
    with_type(x_type, [&](auto t) {
        with_type(y_type, [&](auto r) {
            using T = decltype(t);
            using R = decltype(r);
            // One block of 8 values a thread as long as the SMs hold all threads at once, four where
            // there are more (bf16, one and four: 64 x 4096 1.7 and 2.1 us, 608 x 4096, the border, 3.4
            // and 3.8, 4096 x 4096 14.9 and 14.1).
            const bool few = a.items < 2048 * int64_t(sm_count());
            constexpr int kMany = sizeof(T) + sizeof(R) <= 4 ? 4 : 1;
            if (vec && few) dropout_run<T, R, 1><<<grid(kDropThreads), kDropThreads, 0, stream>>>(a);
            else if (vec) dropout_run<T, R, kMany><<<grid(kDropThreads * kMany), kDropThreads, 0, stream>>>(a);
            else if (lanes == 8) dropout_rows<T, R, 8><<<grid(kDropThreads / 8), kDropThreads, 0, stream>>>(a);
            else if (lanes == 16) dropout_rows<T, R, 16><<<grid(kDropThreads / 16), kDropThreads, 0, stream>>>(a);
            else dropout_rows<T, R, 32><<<grid(kDropThreads / 32), kDropThreads, 0, stream>>>(a);
        });
    });
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace rowops
