// expert_rows.cu - token rows to their experts' slots and back.
//
//   gather       out[slot[t][j]] = x[t]
//   combine      out[t] = sum_j w[t][j] y[slot[t][j]]
//   combine_bwd  dy[slot[t][j]] = w[t][j] dout[t],  dw[t][j] = sum_c dout[t][c] y[slot[t][j]][c]
//
// All three are bound by HBM.  They go token by token, so a token's row is read
// (or written) once however many experts it has, and an expert row is touched
// once; the plan's order decides only where the rows lie.  A slot outside the
// expert matrix is skipped.  Sums are fp32 in the order of the choices (and of
// the columns, for dw), so results repeat bit for bit.  A slot that two pairs name
// is written by both, tile by tile in no fixed order.
//
// Blocks of 128 threads were 2..3% faster than of 256 and 5% faster than of 512;
// combine's rows and results marked to leave the caches first: 19.2 -> 18.0 us (16384 x
// 768 bf16, k = 2; the same marks slow the backward pass, whose dout rows are read
// twice, by 10%).
#include "types.cuh"

namespace rowops {
namespace {

constexpr int kRowThreads = 128;
constexpr int kRowWarps = kRowThreads / 32;

// A group of 2^shift lanes (SHORT; else a warp, which the compiler makes better
// use of) per (token, tile of 2^shift * V * U columns); rows
// shorter than a warp's tile share a warp (64 columns of 262144 tokens, combine:
// 68 -> 33 us, 29 since).
template <typename TI, typename TO, int V, int U, bool SHORT>
__global__ void __launch_bounds__(kRowThreads)
    gather_rows(const TI* __restrict__ x, const int32_t* __restrict__ slot, TO* __restrict__ out, int64_t items,
                int tiles, int shift, int k, int64_t cols, int64_t slots) {
    if constexpr (!SHORT) shift = 5;
    const int lanes = 1 << shift;
    const int64_t item = int64_t(blockIdx.x) * (kRowThreads >> shift) + (threadIdx.x >> shift);
    if (item >= items) return;
    const int64_t t = item / tiles, c0 = (item % tiles) * (lanes * V * U) + (threadIdx.x & (lanes - 1)) * V;
    Chunk<TI, V> in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = c0 + u * (lanes * V);
        if (c < cols) in[u].load(x + t * cols + c);
    }
    Chunk<TO, V> o[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < V; ++i) o[u].set(i, in[u].get(i));
    for (int j = 0; j < k; ++j) {
        const int64_t s = __ldg(slot + t * k + j);
        if (s < 0 || s >= slots) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = c0 + u * (lanes * V);
            if (c < cols) o[u].store(out + s * cols + c);
        }
    }
}

template <typename TI, typename TO, int V, int U, bool SHORT>
__global__ void __launch_bounds__(kRowThreads)
    combine_rows(const TI* __restrict__ y, const int32_t* __restrict__ slot, const float* __restrict__ weights,
                 TO* __restrict__ out, int64_t items, int tiles, int shift, int k, int64_t cols, int64_t slots) {
    if constexpr (!SHORT) shift = 5;
    const int lanes = 1 << shift;
    const int64_t item = int64_t(blockIdx.x) * (kRowThreads >> shift) + (threadIdx.x >> shift);
    if (item >= items) return;
    const int64_t t = item / tiles, c0 = (item % tiles) * (lanes * V * U) + (threadIdx.x & (lanes - 1)) * V;
    float acc[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[u][i] = 0.f;
    for (int j = 0; j < k; ++j) {
        const int64_t s = __ldg(slot + t * k + j);
        if (s < 0 || s >= slots) continue;
        const float w = weights == nullptr ? 1.0f : __ldg(weights + t * k + j);
        Chunk<TI, V> in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = c0 + u * (lanes * V);
            if (c < cols) in[u].load_once(y + s * cols + c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[u][i] = fmaf(w, in[u].get(i), acc[u][i]);
    }
    Chunk<TO, V> o[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = c0 + u * (lanes * V);
#pragma unroll
        for (int i = 0; i < V; ++i) o[u].set(i, acc[u][i]);
        if (c < cols) o[u].store_once(out + t * cols + c);
    }
}

// WARPS warps, or (WARPS == 0) a group of 2^shift lanes, per pair (t, j); pairs of one
// token are neighbours, so its dout row comes from the L1 after the first.  A short
// row's loop makes one or two turns and is not unrolled (262144 x 64: 52.7 -> 41.8 us); the
// others are (4096 x 4096, k = 4: 60.7 -> 55.2 us).
template <typename TO, typename TY, int V, int WARPS>
__global__ void __launch_bounds__(kRowThreads)
    combine_rows_bwd(const TO* __restrict__ dout, const TY* __restrict__ y, const int32_t* __restrict__ slot,
                     const float* __restrict__ weights, TY* __restrict__ dy, float* __restrict__ dweights,
                     int64_t pairs, int shift, int k, int64_t cols, int64_t slots) {
    __shared__ float part[kRowWarps];
    constexpr int kWarps = WARPS > 0 ? WARPS : 1;
    if constexpr (WARPS > 0) shift = 5;
    const int warp = threadIdx.x >> 5, lanes = 1 << shift, lane = threadIdx.x & (lanes - 1);
    const int64_t p = WARPS > 0 ? int64_t(blockIdx.x) * (kRowWarps / kWarps) + warp / kWarps
                                : int64_t(blockIdx.x) * (kRowThreads >> shift) + (threadIdx.x >> shift);
    const int64_t s = p < pairs ? int64_t(__ldg(slot + p)) : -1;
    float dot = 0.f;
    if (s >= 0 && s < slots) {
        const float w = __ldg(weights + p);
        const TO* d = dout + (p / k) * cols;
#pragma unroll (WARPS > 0 ? 4 : 1)
        for (int64_t c = ((WARPS > 0 ? warp % kWarps : 0) * lanes + lane) * V; c < cols; c += kWarps * lanes * V) {
            Chunk<TO, V> a;
            Chunk<TY, V> b, o;
            a.load(d + c);
            b.load(y + s * cols + c);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dot = fmaf(a.get(i), b.get(i), dot);
                o.set(i, w * a.get(i));
            }
            o.store(dy + s * cols + c);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < lanes) dot += __shfl_xor_sync(kFullMask, dot, o);
    if constexpr (WARPS > 1) {
        if (lane == 0) part[warp] = dot;
        __syncthreads();
        if (threadIdx.x == 0 && p < pairs) {
            float sum = part[0];
            for (int i = 1; i < WARPS; ++i) sum += part[i];
            dweights[p] = sum;
        }
    } else if (lane == 0 && p < pairs) {
        dweights[p] = dot;
    }
}

bool chunked(const void* p, int64_t cols, int v, size_t size) {
    return cols % v == 0 && reinterpret_cast<uintptr_t>(p) % (v * size) == 0;
}

// Lanes of a group that covers `cols` columns with `per` columns a lane: a power of two up to 32.
int group_shift(int64_t cols, int per) {
    int shift = 0;
    while (shift < 5 && (int64_t(per) << shift) < cols) ++shift;
    return shift;
}

struct Items {
    int64_t items;
    int tiles, shift;
    unsigned grid;
};
inline Items row_items(int64_t rows, int64_t cols, int per) {
    Items r;
    r.shift = group_shift(cols, per);
    const int64_t tile = int64_t(per) << r.shift;
    r.tiles = int((cols + tile - 1) / tile);
    r.items = rows * r.tiles;
    const int64_t block = kRowThreads >> r.shift;
    r.grid = unsigned((r.items + block - 1) / block);
    return r;
}

}  // namespace

cudaError_t launch_expert_gather(const void* x, const int32_t* slot, void* out, int64_t rows, int64_t k,
                                 int64_t cols, int64_t slots, int x_type, int out_type, cudaStream_t stream) {
    with_type(x_type, [&](auto ti) {
        with_type(out_type, [&](auto to) {
            using TI = decltype(ti);
            using TO = decltype(to);
            constexpr int V = chunk_of<TI, TO>();
            const TI* xp = static_cast<const TI*>(x);
            TO* op = static_cast<TO*>(out);
            auto go = [&](auto kernel, const Items& n) {
                kernel<<<n.grid, kRowThreads, 0, stream>>>(xp, slot, op, n.items, n.tiles, n.shift, int(k), cols, slots);
            };
            if (chunked(x, cols, V, sizeof(TI)) && chunked(out, cols, V, sizeof(TO))) {
                const Items n = row_items(rows, cols, V * 2);
                if (n.shift < 5) go(gather_rows<TI, TO, V, 2, true>, n);
                else go(gather_rows<TI, TO, V, 2, false>, n);
            } else {
                const Items n = row_items(rows, cols, 4);
                if (n.shift < 5) go(gather_rows<TI, TO, 1, 4, true>, n);
                else go(gather_rows<TI, TO, 1, 4, false>, n);
            }
        });
    });
    note_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_expert_combine(const void* y, const int32_t* slot, const float* weights, void* out, int64_t rows,
                                  int64_t k, int64_t cols, int64_t slots, int y_type, int out_type,
                                  cudaStream_t stream) {
    with_type(y_type, [&](auto ti) {
        with_type(out_type, [&](auto to) {
            using TI = decltype(ti);
            using TO = decltype(to);
            constexpr int V = chunk_of<TI, TO>();
            const TI* yp = static_cast<const TI*>(y);
            TO* op = static_cast<TO*>(out);
            auto go = [&](auto kernel, const Items& n) {
                kernel<<<n.grid, kRowThreads, 0, stream>>>(yp, slot, weights, op, n.items, n.tiles, n.shift, int(k), cols,
                                                           slots);
            };
            if (chunked(y, cols, V, sizeof(TI)) && chunked(out, cols, V, sizeof(TO))) {
                const Items n = row_items(rows, cols, V * 2);
                if (n.shift < 5) go(combine_rows<TI, TO, V, 2, true>, n);
                else go(combine_rows<TI, TO, V, 2, false>, n);
            } else {
                const Items n = row_items(rows, cols, 4);
                if (n.shift < 5) go(combine_rows<TI, TO, 1, 4, true>, n);
                else go(combine_rows<TI, TO, 1, 4, false>, n);
            }
        });
    });
    note_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_expert_combine_bwd(const void* dout, const void* y, const int32_t* slot, const float* weights,
                                      void* dy, float* dweights, int64_t rows, int64_t k, int64_t cols,
                                      int64_t slots, int out_type, int y_type, cudaStream_t stream) {
    const int64_t pairs = rows * k;
    // Few pairs: a block each, more a warp each (block against warp, 768 columns: 1024 pairs
    // 2.53 and 2.68 us, 2048 4.42 and 4.97, 4096 7.10 and 6.19, 8192 11.8 and 10.3; 4096 columns: 256 pairs
    // 3.65 and 7.01 us, 2048 10.0 and 14.3, 8192 31.9 and 36.8).
    const bool wide = pairs < 16 * int64_t(sm_count());
    with_type(out_type, [&](auto to) {
        with_type(y_type, [&](auto ty) {
            using TO = decltype(to);
            using TY = decltype(ty);
            constexpr int V = chunk_of<TO, TY>();
            const bool vec = chunked(dout, cols, V, sizeof(TO)) && chunked(y, cols, V, sizeof(TY)) &&
                             chunked(dy, cols, V, sizeof(TY));
            const int shift = group_shift(cols, vec ? V * 2 : 4);
            auto go = [&](auto kernel, int warps) {
                const int64_t per = warps > 0 ? kRowWarps / warps : kRowThreads >> shift;
                kernel<<<unsigned((pairs + per - 1) / per), kRowThreads, 0, stream>>>(
                    static_cast<const TO*>(dout), static_cast<const TY*>(y), slot, weights, static_cast<TY*>(dy),
                    dweights, pairs, shift, int(k), cols, slots);
            };
            if (vec && wide) go(combine_rows_bwd<TO, TY, V, kRowWarps>, kRowWarps);
            else if (vec && shift < 5) go(combine_rows_bwd<TO, TY, V, 0>, 0);
            else if (vec) go(combine_rows_bwd<TO, TY, V, 1>, 1);
            else if (wide) go(combine_rows_bwd<TO, TY, 1, kRowWarps>, kRowWarps);
            else if (shift < 5) go(combine_rows_bwd<TO, TY, 1, 0>, 0);
            else go(combine_rows_bwd<TO, TY, 1, 1>, 1);
        });
    });
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace rowops
