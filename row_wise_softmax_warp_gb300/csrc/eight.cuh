// eight.cuh - rows held eight values a lane, for rows of any length and alignment.
//
// A group of LANES lanes holds 8 * LANES neighbouring columns of a row.  VEC (rows
// on 16-byte boundaries, columns a multiple of 8): lane g holds columns 8g .. 8g + 7,
// moved by 16-byte accesses.  Otherwise lane g holds columns g, LANES + g, 2 LANES + g,
// ..., so that each of its eight accesses lies beside its neighbours'.
//
// Blocks of 8 columns (of the generator), of 32 and of 128 (of the quantisers) lie
// inside a group either way.
#pragma once

#include "philox.cuh"
#include "types.cuh"

namespace rowops {

// Eight values as loaded: 16-bit ones take four registers until they are used.
// Loads are not of the read-only kind: an output may be the input's buffer.
template <typename T, int LANES, bool VEC>
struct Held;
template <typename T, int LANES>
struct Held<T, LANES, true> {
    static constexpr int V = 16 / int(sizeof(T));
    Chunk<T, V> c[8 / V];
    __device__ __forceinline__ void load(const T* row, int base, int g, int cols) {
        if (base + 8 * g < cols) {
#pragma unroll
            for (int h = 0; h < 8 / V; ++h) c[h].load_once(row + base + 8 * g + h * V);
        } else {
#pragma unroll
            for (int h = 0; h < 8 / V; ++h) c[h] = Chunk<T, V>();
        }
    }
    __device__ __forceinline__ float get(int i) const { return c[i / V].get(i % V); }
};
template <typename T, int LANES>
struct Held<T, LANES, false> {
    T v[8];
    __device__ __forceinline__ void load(const T* row, int base, int g, int cols) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = base + i * LANES + g;
            v[i] = c < cols ? row[c] : from_float<T>(0.f);
        }
    }
    __device__ __forceinline__ float get(int i) const { return to_float(v[i]); }
};

template <int LANES, bool VEC, typename T>
__device__ __forceinline__ void store_eight(T* row, int base, int g, int cols, const float (&v)[8]) {
    if constexpr (VEC) {
        constexpr int V = 16 / int(sizeof(T));
        if (base + 8 * g < cols) {
#pragma unroll
            for (int h = 0; h < 8 / V; ++h) {
                Chunk<T, V> c;
#pragma unroll
                for (int i = 0; i < V; ++i) c.set(i, v[h * V + i]);
                c.store(row + base + 8 * g + h * V);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = base + i * LANES + g;
            if (c < cols) row[c] = from_float<T>(v[i]);
        }
    }
}

// Parameters: read by every row, so they stay in the caches.
template <int LANES, bool VEC>
__device__ __forceinline__ void load_weights(const float* p, int base, int g, int cols, float (&v)[8]) {
    if constexpr (VEC) {
        float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
        if (base + 8 * g < cols) {
            ld_chunk<4>(p + base + 8 * g, a);
            ld_chunk<4>(p + base + 8 * g + 4, b);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = base + i * LANES + g;
            v[i] = c < cols ? __ldg(p + c) : 0.f;
        }
    }
}

// v with values dropped and the others scaled.  The whole warp calls it, every group
// for a row of its own.  per: blocks of 8 in a row.  What drops is +0.0 whatever it was.
template <int LANES, bool VEC>
__device__ __forceinline__ void drop_eight(float (&v)[8], const Dropout& d, const Masker& m, int64_t row, int per,
                                           int base, int g) {
    if (d.threshold == 0) return;
    if (d.threshold == 65536) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
        return;
    }
    bool keep[8];
    m.block(uint64_t(row) * uint32_t(per) + uint32_t(base / 8 + g), keep);
    if constexpr (!VEC) {  // lane g made block g of the group; value i of it is of block i * LANES / 8 + g / 8
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) bits |= uint32_t(keep[i]) << i;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            keep[i] = (__shfl_sync(kFullMask, bits, i * (LANES / 8) + g / 8, LANES) >> (g & 7)) & 1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = keep[i] ? v[i] * d.scale : 0.f;
}

// How a kernel walks its rows: `warps` warps hold one (LANES lanes where it is
// short), `slots` such sets of warps are in a block.
struct RowSplit {
    int warps, slots;
};

// The sum over the row that this lane's group or set of warps holds.  scratch: a
// float a warp of the block, of a buffer that the last call did not use.
template <int LANES>
__device__ __forceinline__ float sum_of_row(float v, float* scratch, int warps, int slot, int w) {
    v = group_sum<LANES>(v);
    if (LANES < 32 || warps == 1) return v;
    scratch += slot * warps;
    const int lane = threadIdx.x & 31;
    if (lane == 0) scratch[w] = v;
    asm volatile("bar.sync %0, %1;\n" ::"r"(slot + 1), "r"(warps * 32) : "memory");  // slot + 1 <= 15
    return group_sum<32>(lane < warps ? scratch[lane] : 0.f);
}

// Host: f(T{}, R{}) for the types of a branch and of its residual stream, which is
// of the same type or fp32.
template <typename F>
bool with_branch_types(int x_type, int h_type, F&& f) {
    if (x_type == ROWOPS_F32 && h_type == ROWOPS_F32) f(float{}, float{});
    else if (x_type == ROWOPS_F16 && h_type == ROWOPS_F16) f(__half{}, __half{});
    else if (x_type == ROWOPS_F16 && h_type == ROWOPS_F32) f(__half{}, float{});
    else if (x_type == ROWOPS_BF16 && h_type == ROWOPS_BF16) f(__nv_bfloat16{}, __nv_bfloat16{});
    else if (x_type == ROWOPS_BF16 && h_type == ROWOPS_F32) f(__nv_bfloat16{}, float{});
    else return false;
    return true;
}

}  // namespace rowops
