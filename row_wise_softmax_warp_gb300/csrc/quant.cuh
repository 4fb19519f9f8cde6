// quant.cuh - e4m3 values with a scale for a block, and e2m1 values with a power of two.
#pragma once

#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace rowops {

constexpr float kLargest = 448.0f;        // of e4m3
constexpr float kSmallestMax = 0x1p-100f;

// Largest magnitude; NaN values do not count, infinite ones do.
__device__ __forceinline__ float largest(const float (&v)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}
// Largest finite magnitude.
__device__ __forceinline__ float largest_finite(const float (&v)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (fabsf(v[i]) < INFINITY) m = fmaxf(m, fabsf(v[i]));
    return m;
}

// a / 448, correctly rounded: the same step with the rounded reciprocal of 448.
__device__ __forceinline__ float scale_of(float a) {
    constexpr float kInv = 1.0f / kLargest;
    const float q0 = a * kInv;
    return fmaf(fmaf(-q0, kLargest, a), kInv, q0);
}

// 448 x / a by the reciprocal and one residual step (Markstein 1990): q0 is off by
// at most three units, r is its exact residual, and a quotient that fp32 holds (as
// every border between e4m3 values does) comes out exact.  An infinite or NaN x
// makes r NaN.  x and a are divided by 2^32 where 448 x could overflow.
struct Divisor {
    float scale, d, inv;
    __device__ __forceinline__ explicit Divisor(float a) {
        const float s = a > 0x1p100f ? 0x1p-32f : 1.0f;
        scale = kLargest * s;
        d = a * s;
        asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(inv) : "f"(d));  // off by a unit at most
    }
    __device__ __forceinline__ float operator()(float x) const {
        const float t = x * scale, q0 = t * inv, r = fmaf(-q0, d, t);
        return fmaf(r, inv, q0);
    }
};

__device__ __forceinline__ uint2 quantize8(const float (&v)[8], const Divisor& over) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(over(v[2 * i]), over(v[2 * i + 1])), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// ------------------------------------------------- microscaled 4 bits (e2m1, e8m0)
//
// A block of 32 shares 2^(code - 127) with code - 127 = floor(log2 a) - 2 (2: the
// exponent of 6, the largest e2m1), at least -127: OCP Microscaling Formats 1.0, 6.3.
// Values past 6 after the division become 6.  A block with an infinite or NaN value has
// code 255, which stands for NaN, and zeros.

// The largest magnitude as its bits, in which NaN lies above infinity.
__device__ __forceinline__ uint32_t largest_bits(const float2 (&v)[4]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = max(m, max(__float_as_uint(v[i].x) & 0x7fffffffu, __float_as_uint(v[i].y) & 0x7fffffffu));
    return m;
}
template <int LANES>
__device__ __forceinline__ uint32_t group_max_bits(uint32_t v) {
    if constexpr (LANES == 32) {
        return __reduce_max_sync(kFullMask, v);
    } else {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFullMask, v, o));
        return v;
    }
}
// The block's code from its largest magnitude.  A subnormal's exponent field is 0, and
// floor(log2 a) - 2 lies below -127 for it.
__device__ __forceinline__ uint32_t mx4_code(uint32_t bits) {
    const uint32_t e = bits >> 23;
    return e == 255 ? 255 : max(int(e) - 2, 0);
}
// 2^(127 - code), by which a block's values are multiplied: exact but where the result is
// far below the least e2m1.  0 for code 255.
__device__ __forceinline__ float mx4_inverse(uint32_t code) {
    return code == 255 ? 0.f : __uint_as_float((254 - code) << 23);
}
// Two codes in a byte, the first value in the lower half; 0 times an infinite or NaN value
// would be NaN, so blocks of code 255 are told.
__device__ __forceinline__ uint32_t mx4_pair(float2 v, float inverse) {
    return __nv_cvt_float2_to_fp4x2(make_float2(v.x * inverse, v.y * inverse), __NV_E2M1, cudaRoundNearest);
}
__device__ __forceinline__ uint32_t mx4_eight(const float2 (&v)[4], uint32_t code) {
    if (code == 255) return 0;
    const float inverse = mx4_inverse(code);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= mx4_pair(v[i], inverse) << (8 * i);
    return w;
}

// ----------------------------------------------------- quantised columns of a row
//
// Eight values of each lane of a group, placed as in eight.cuh, to their row of bytes and
// of scales.  The whole warp calls them.  Blocks of 128 columns are 16 lanes' (VEC; or the
// whole of a shorter group), or four values of each of 32 lanes.

template <int LANES, bool VEC>
__device__ __forceinline__ void store_e4m3(uint8_t* q, float* scale, int base, int g, int cols, const float2 (&pairs)[4]) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[2 * i] = pairs[i].x, y[2 * i + 1] = pairs[i].y;
    scale += base / 128;
    if constexpr (VEC) {
        constexpr int kBlock = LANES < 16 ? LANES : 16;
        float most = group_max<kBlock>(largest(y));
        if (__any_sync(kFullMask, most == INFINITY)) most = group_max<kBlock>(largest_finite(y));
        most = fmaxf(most, kSmallestMax);
        if (base + 8 * g < cols) {
            *reinterpret_cast<uint2*>(q + base + 8 * g) = quantize8(y, Divisor(most));
            if (g % kBlock == 0) scale[g / kBlock] = scale_of(most);
        }
    } else {
        static_assert(LANES == 32, "a value of each lane is 32 columns");
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint32_t most = 0, fine = 0;  // as bits; NaN does not count
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = fmaxf(fabsf(y[b * 4 + i]), 0.f);
                most = max(most, __float_as_uint(v));
                if (v < INFINITY) fine = max(fine, __float_as_uint(v));
            }
            float a = __uint_as_float(group_max_bits<32>(most));
            if (a == INFINITY) a = __uint_as_float(group_max_bits<32>(fine));  // the same in all lanes
            a = fmaxf(a, kSmallestMax);
            const Divisor over(a);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = base + (b * 4 + i) * 32 + g;
                if (c < cols) q[c] = __nv_cvt_float_to_fp8(over(y[b * 4 + i]), __NV_SATFINITE, __NV_E4M3);
            }
            if (g == 0 && base + b * 128 < cols) scale[b] = scale_of(a);
        }
    }
}

template <int LANES, bool VEC>
__device__ __forceinline__ void store_mx4(uint8_t* q, uint8_t* scale, int base, int g, int cols, const float2 (&pairs)[4]) {
    scale += base / 32;
    if constexpr (VEC) {
        const uint32_t code = mx4_code(group_max_bits<4>(largest_bits(pairs)));
        if (base + 8 * g < cols) {
            *reinterpret_cast<uint32_t*>(q + base / 2 + 4 * g) = mx4_eight(pairs, code);
            if (g % 4 == 0) scale[g / 4] = uint8_t(code);
        }
    } else {
        static_assert(LANES == 32, "a value of each lane is a block");
        uint32_t code[8];
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[2 * i] = pairs[i].x, y[2 * i + 1] = pairs[i].y;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            code[i] = mx4_code(group_max_bits<32>(__float_as_uint(y[i]) & 0x7fffffffu));
            if (g == 0 && base + i * 32 < cols) scale[i] = uint8_t(code[i]);
        }
        // Of two blocks, even lanes write the first's bytes, odd lanes the second's.
        const bool odd = g & 1;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float other = __shfl_xor_sync(kFullMask, odd ? y[i] : y[i + 1], 1);
            const uint32_t mine = odd ? code[i + 1] : code[i];
            const int c = base + (i + odd) * 32 + g - odd;
            if (c < cols)
                q[c / 2] = mine == 255 ? 0 : uint8_t(mx4_pair(make_float2(odd ? other : y[i], odd ? y[i + 1] : other), mx4_inverse(mine)));
        }
    }
}

}  // namespace rowops
