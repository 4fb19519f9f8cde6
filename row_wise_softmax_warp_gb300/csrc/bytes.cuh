// bytes.cuh - bytes that start anywhere, read by aligned words.
#pragma once

#include <cstdint>

namespace rowops {

// N aligned words from `at`, of whose bytes those in [begin, end) are there; the others
// are 0.  The words that lie inside are asked for together; the first and the last of all,
// which may be there in part, are put together once, by bytes (per word, the code of that
// alone took the scales of a 4-bit product 3 us to fetch).  Plain loads: programmatic
// dependents read what was written after they began.
__device__ __forceinline__ uint32_t part_of_word(const uint8_t* at, const uint8_t* begin, const uint8_t* end) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (at + i >= begin && at + i < end) w |= uint32_t(at[i]) << (8 * i);
    return w;
}
template <int N>
__device__ __forceinline__ void words_at(const uint8_t* at, const uint8_t* begin, const uint8_t* end, uint32_t (&w)[N]) {
    const int64_t there = end - at;
    const int whole = there >= 4 * N ? N : there > 0 ? int(there) >> 2 : 0;
    const bool front = at >= begin;
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = i < whole && (i > 0 || front) ? reinterpret_cast<const uint32_t*>(at)[i] : 0;
    if (!front || whole < N) {
        const uint32_t last = part_of_word(at + 4 * whole, begin, end);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i == whole) w[i] = last;
        if (!front) w[0] = part_of_word(at, begin, end);
    }
}

}  // namespace rowops
