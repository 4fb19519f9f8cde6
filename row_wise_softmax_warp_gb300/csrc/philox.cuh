// philox.cuh - the counter-based generator of the dropout operators.
//
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as
// 1, 2, 3; SC 2011): ten rounds of two 32 x 32-bit products on a 128-bit counter.
// A row of `cols` values has ceil(cols / 8) blocks of 8; block j of the matrix takes
// the 128 bits of the counter (j, rng[1]) under the key rng[0], 16 for each value.
// So a mask is a function of rng, the row and the column alone: the backward pass
// makes it again, and nothing of it is stored.  Sixteen bits a value halve the
// products of 32; a probability is then rounded to a multiple of 2^-16, and the scale
// of what is kept goes by the rounded one.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace rowops {

struct Dropout {
    const uint64_t* rng;  // key and offset; read only where threshold is 1 .. 65535
    int threshold;        // 0: nothing drops; 65536: everything
    float scale;
};
inline Dropout dropout_of(const uint64_t* rng, float p) {
    const int t = dropout_threshold(p);
    return {rng, t, dropout_scale(t)};
}

// The generator with its key and offset loaded.
struct Masker {
    uint32_t k0, k1, c2, c3, limit;

    __device__ __forceinline__ explicit Masker(const Dropout& d) : k0(0), k1(0), c2(0), c3(0), limit(0) {
        if (d.threshold == 0 || d.threshold == 65536) return;
        const uint64_t key = __ldg(d.rng), offset = __ldg(d.rng + 1);
        k0 = uint32_t(key);
        k1 = uint32_t(key >> 32);
        c2 = uint32_t(offset);
        c3 = uint32_t(offset >> 32);
        limit = uint32_t(d.threshold) << 16;
    }
    // keep[i]: value i of block j stays
    __device__ __forceinline__ void block(uint64_t j, bool (&keep)[8]) const {
        uint32_t a = uint32_t(j), b = uint32_t(j >> 32), c = c2, d = c3, k = k0, l = k1;
#pragma unroll
        for (int r = 0; r < 10; ++r) {
            const uint64_t m = uint64_t(a) * 0xD2511F53u, n = uint64_t(c) * 0xCD9E8D57u;
            a = uint32_t(n >> 32) ^ b ^ k;
            b = uint32_t(n);
            c = uint32_t(m >> 32) ^ d ^ l;
            d = uint32_t(m);
            k += 0x9E3779B9u;
            l += 0xBB67AE85u;
        }
        const uint32_t w[4] = {a, b, c, d};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            keep[2 * i] = (w[i] << 16) >= limit;
            keep[2 * i + 1] = w[i] >= limit;
        }
    }
};

}  // namespace rowops
