// row_store.cuh - results that lie a row a lane, written in whole lines.
//
// Tensor memory gives lane i row i.  Written from there, each 16-byte store of a
// warp touches 32 lines; turned in shared memory first, it touches 4 of 128 bytes
// (32768 rows, 16 experts, 2048 x 4096: e4m3 product 326 -> 279 us; 16384 x 4096 x
// 4096 e4m3: 254 -> 230 us; 64 experts of 768 x 2048: weights' gradient 98 -> 65 us).
#pragma once

#include "types.cuh"

namespace rowops {

constexpr int kTurnBytes = 32 * 128;  // of shared memory per warp, 16-byte aligned

// One warp writes 128 bytes (COLS values) of 32 rows: lane i holds row i's values
// v(0) .. v(COLS - 1).  p: first value of row 0; pitch: values from row to row; rows,
// cols: what is there.  vec: p, pitch and cols are multiples of 16 bytes; else the
// lines are written value by value.
template <typename O, typename F>
__device__ __forceinline__ void store_rows(unsigned char* turn, O* p, int64_t pitch, int rows, int cols, bool vec, F&& v) {
    constexpr int V = 16 / int(sizeof(O));
    const int lane = threadIdx.x & 31;
    __syncwarp();  // the last use's reads are done
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        Chunk<O, V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) o.set(i, v(j * V + i));
        o.store(reinterpret_cast<O*>(turn + lane * 128 + ((j ^ (lane & 7)) * 16)));  // no two lanes in a bank
    }
    __syncwarp();
    if (!vec) {
        constexpr int kCols = 128 / int(sizeof(O));
        for (int row = 0; row < min(rows, 32); ++row)
#pragma unroll
            for (int c = lane; c < kCols; c += 32)
                if (c < cols)
                    p[row * pitch + c] =
                        reinterpret_cast<const O*>(turn + row * 128 + ((c / V) ^ (row & 7)) * 16)[c % V];
        return;
    }
    const int chunk = lane & 7;
    if (chunk * V < cols) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = i * 4 + (lane >> 3);
            if (row < rows)
                *reinterpret_cast<uint4*>(p + row * pitch + chunk * V) =
                    *reinterpret_cast<const uint4*>(turn + row * 128 + ((chunk ^ (row & 7)) * 16));
        }
    }
}

}  // namespace rowops
