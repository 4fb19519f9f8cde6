// Test-only: the experts' table of tiles by itself, without any matrix, so that
// groups of up to 2^30 rows can be looked at.
#include "groups.cuh"

using namespace rowops;

extern "C" unsigned host_tiles_of(int rows, int tile) { return tiles_of(rows, tile); }
extern "C" int host_cut_tiles(unsigned n) { return cut_tiles(n); }
extern "C" int host_all_tiles(int row_tiles, int across) { return all_tiles(row_tiles, across); }

// table[experts + 1]; for each of `n` row tiles: expert, first row, rows.
template <int NT>
__global__ void __launch_bounds__(NT)
    tile_probe(const int32_t* offsets, int experts, int slots, int* table_out, const int* asked, int n, int* out) {
    __shared__ int table[kMaxExperts + 1], scratch[NT / 32];
    build_tile_table<kMostRows, NT>(offsets, experts, slots, table, scratch);
    __syncthreads();
    for (int e = threadIdx.x; e <= experts; e += NT) table_out[e] = table[e];
    if (threadIdx.x >= 32) return;
    int from = 0;
    for (int i = 0; i < n; ++i) {
        const int tile = asked[i];
        if (tile < 0 || tile >= table[experts]) continue;
        const RowTile t = row_tile(offsets, experts, slots, table, tile, from);
        from = t.expert;
        if (threadIdx.x == 0) {
            out[3 * i] = t.expert;
            out[3 * i + 1] = t.first;
            out[3 * i + 2] = t.count;
        }
    }
}

extern "C" int run_tile_probe(int threads, const int32_t* offsets, int experts, int slots, int* table, const int* asked,
                              int n, int* out) {
    if (experts < 1 || experts > kMaxExperts) return -1;
    if (threads == 224) tile_probe<224><<<1, 224>>>(offsets, experts, slots, table, asked, n, out);
    else if (threads == 384) tile_probe<384><<<1, 384>>>(offsets, experts, slots, table, asked, n, out);
    else return -1;
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? int(e) : int(cudaDeviceSynchronize());
}
