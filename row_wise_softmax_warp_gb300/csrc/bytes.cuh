// bytes.cuh - bytes that start anywhere, read by aligned words.
#pragma once

#include <cstdint>

namespace rowops {

// The aligned word at `at`, of whose bytes those in [begin, end) are there.  A plain load:
// programmatic dependents read what was written after they began.
__device__ __forceinline__ uint32_t word_at(const uint8_t* at, const uint8_t* begin, const uint8_t* end) {
    if (at >= begin && at + 4 <= end) return *reinterpret_cast<const uint32_t*>(at);
    uint32_t w = 0;
    for (int i = 0; i < 4; ++i)
        if (at + i >= begin && at + i < end) w |= uint32_t(at[i]) << (8 * i);
    return w;
}

}  // namespace rowops
