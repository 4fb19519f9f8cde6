// groups.cuh - rows grouped by expert: expert e owns rows offsets[e] ..
// offsets[e + 1] - 1 of a matrix of `slots` rows.
//
// The offsets are device data that no host check has seen, so every read of
// them is clamped to 0 .. slots with ends not before starts: bad offsets give
// wrong rows, never an access out of bounds.
#pragma once

#include "common.cuh"

namespace rowops {

constexpr int kMaxExperts = 1024;

// Groups that overlap (offsets that fall and rise again: bad ones, but stay in
// bounds) can name every row up to 512 times, so counts of tiles are added up
// unsigned, which holds 512 * 2^30 rows in tiles of more than 128, and cut at kMostTiles.
// Groups that do not overlap have fewer: the host refuses more than kMostTiles.
constexpr int kMostTiles = 1 << 30;

__host__ __device__ constexpr unsigned tiles_of(int rows, int tile) { return unsigned(rows / tile + (rows % tile != 0)); }
__host__ __device__ constexpr int cut_tiles(unsigned n) { return n < unsigned(kMostTiles) ? int(n) : kMostTiles; }
// Tiles of `row_tiles` rows of tiles, `across` each: a tile's number plus a grid stays in 32 bits.
__host__ __device__ constexpr int all_tiles(int row_tiles, int across) {
    const int64_t n = int64_t(row_tiles) * across;
    return n < kMostTiles ? int(n) : kMostTiles;
}

struct RowRange {
    int first, count;
};

__device__ __forceinline__ RowRange group_rows(const int32_t* offsets, int e, int slots) {
    if (offsets == nullptr) return {0, slots};  // one dense group
    const int lo = min(max(offsets[e], 0), slots);  // plain loads: a programmatic dependent reads them too
    const int hi = min(max(offsets[e + 1], lo), slots);
    return {lo, hi - lo};
}

// Expert, first row and row count of row tile `tile` (tiles of TILE rows,
// counted over the experts in order); false past the last tile.  Called by a
// whole warp, which scans the experts 32 at a time.
template <int TILE>
__device__ __forceinline__ bool find_row_tile(const int32_t* offsets, int experts, int slots, int64_t tile,
                                              int& expert, int& first, int& count) {
    const int lane = threadIdx.x & 31;
    int64_t before = 0;
    for (int base = 0; base < experts; base += 32) {
        const int e = base + lane;
        RowRange r{0, 0};
        if (e < experts) r = group_rows(offsets, e, slots);
        const int n = int(tiles_of(r.count, TILE));
        int upto = n;  // inclusive scan over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFullMask, upto, o);
            if (lane >= o) upto += v;
        }
        const unsigned past = __ballot_sync(kFullMask, before + upto > tile);
        if (past) {
            const int src = __ffs(past) - 1;
            const int in_group = int(tile - before) - (__shfl_sync(kFullMask, upto, src) - __shfl_sync(kFullMask, n, src));
            const int at = in_group * TILE;
            expert = base + src;
            first = __shfl_sync(kFullMask, r.first, src) + at;
            count = min(TILE, __shfl_sync(kFullMask, r.count, src) - at);
            return true;
        }
        before += __shfl_sync(kFullMask, upto, 31);
    }
    return false;
}

// table[e] = row tiles of the experts before e (table[experts]: all), cut at kMostTiles.
// Called by the whole block, which synchronises before the table is read; scratch: an int a warp.
// keep(expert, rows, tiles) is called by the thread that looked the expert's rows up.
struct KeepNothing {
    __device__ __forceinline__ void operator()(int, const RowRange&, unsigned) const {}
};
template <int TILE, int NT, typename Keep = KeepNothing>
__device__ __forceinline__ void build_tile_table(const int32_t* offsets, int experts, int slots, int* table,
                                                 int* scratch, Keep keep = Keep()) {
    static_assert(TILE > 128, "512 groups of 2^30 rows have to fit the sum");
    constexpr int kPer = (kMaxExperts + NT - 1) / NT;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (experts + NT - 1) / NT, first = threadIdx.x * per;  // a run of experts each
    unsigned n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        n[i] = 0;
        if (i < per && first + i < experts) {
            const RowRange r = group_rows(offsets, first + i, slots);
            n[i] = tiles_of(r.count, TILE);
            keep(first + i, r, n[i]);
        }
        sum += n[i];
    }
    unsigned upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(kFullMask, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) scratch[warp] = int(upto);
    __syncthreads();
    unsigned before = upto - sum;
    for (int w = 0; w < warp; ++w) before += unsigned(scratch[w]);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (i < per && first + i < experts) table[first + i] = cut_tiles(before);
        before += n[i];
    }
    if (threadIdx.x == NT - 1) table[experts] = cut_tiles(before);
}

// The expert of row tile `tile`, 0 <= tile < table[experts], for tiles asked for in
// rising order: from is the last answer (0 at first).  The whole warp looks at 32
// experts at once: a binary search in shared memory would wait for six looks, one
// after another, before every tile (64 experts, 768 -> 2048, e4m3, 8192 rows: 47 us; so 46).
__device__ __forceinline__ int tile_expert(const int* table, int experts, int tile, int from) {
    const int lane = threadIdx.x & 31;
    for (int e = from;; e += 32) {
        const int next = e + 1 + lane;  // table[next] <= tile: the tile lies behind expert next - 1
        const unsigned behind = __ballot_sync(kFullMask, next <= experts && table[next] <= tile);
        if (behind != 0xffffffffu) return e + __popc(behind);
    }
}

// Groups cut into even tiles for the tcgen05 products: a group of n rows into
// ceil(n / kMostRows) tiles of a multiple of 32 rows (the last may be shorter).
constexpr int kMostRows = 256;

struct RowTile {
    int expert, first, count;
};

// table: build_tile_table<kMostRows>; 0 <= tile < table[experts], and from as for tile_expert.
__device__ __forceinline__ RowTile row_tile(const int32_t* offsets, int experts, int slots, const int* table,
                                            int tile, int from) {
    RowTile t;
    t.expert = tile_expert(table, experts, tile, from);
    const RowRange r = group_rows(offsets, t.expert, slots);
    const int tiles = (r.count + kMostRows - 1) / kMostRows;
    const int each = ((r.count + tiles - 1) / tiles + 31) & ~31;  // at most kMostRows, and every tile gets a row
    const int at = (tile - table[t.expert]) * each;
    t.first = r.first + at;
    t.count = min(each, r.count - at);
    return t;
}

// The same from shared memory: what a tile needs of its group is worked out once, by the
// thread that builds the table, so that a tile is found without a look at memory or a
// division (a warp alone took 1300 clocks for its first tile, so some 250).
struct Group {
    int first, count, each;  // rows, and those of a tile
};
template <int MOST>
struct KeepGroups {
    static_assert(MOST % 32 == 0 && MOST > 128, "even tiles of a multiple of 32 rows are no more than MOST");
    Group* groups;
    __device__ __forceinline__ void operator()(int e, const RowRange& r, unsigned tiles) const {
        const int n = tiles > 1 ? int((unsigned(r.count) + tiles - 1) / tiles) : r.count;
        groups[e] = {r.first, r.count, (n + 31) & ~31};
    }
};
// table: build_tile_table<MOST> with KeepGroups<MOST>
__device__ __forceinline__ RowTile kept_row_tile(const Group* groups, int experts, const int* table, int tile, int from) {
    RowTile t;
    t.expert = tile_expert(table, experts, tile, from);
    const Group r = groups[t.expert];
    const int at = (tile - table[t.expert]) * r.each;
    t.first = r.first + at;
    t.count = min(r.each, r.count - at);
    return t;
}

// Host: the most row tiles that groups of `slots` rows in all can have.
inline int64_t most_row_tiles(int64_t slots, int64_t experts, int most = kMostRows) {
    return slots / most + (experts < slots ? experts : slots);
}

}  // namespace rowops
