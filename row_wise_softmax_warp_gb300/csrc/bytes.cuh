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
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint8_t* p = at + 4 * i;
        w[i] = p >= begin && p + 4 <= end ? *reinterpret_cast<const uint32_t*>(p) : 0;
    }
    if (at < begin) {
        const uint8_t* first = begin - (reinterpret_cast<uintptr_t>(begin) & 3);
        const uint32_t part = part_of_word(first, begin, end);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (at + 4 * i == first) w[i] = part;
    }
    const uint8_t* last = end - (reinterpret_cast<uintptr_t>(end) & 3);
    if (last < end && at + 4 * N > last) {
        const uint32_t part = part_of_word(last, begin, end);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (at + 4 * i == last) w[i] = part;
    }
}

}  // namespace rowops
