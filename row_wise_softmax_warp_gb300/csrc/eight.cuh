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

// Pairs of fp32 values: one instruction for two of each operation.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Two 16-bit values in a word, the first in its lower half.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float2 v);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float2 v) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&p);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float2 v) {
    const __half2 p = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// A lane's eight values: the index of the first, and how many columns there are from it to
// the row's end (none: 0 or less).  VEC: the next seven are its neighbours; else they lie
// LANES apart.
template <int LANES, bool VEC>
struct Place {
    int64_t at;
    int left;
    // there: columns of the row that are there, 0 for a row that is not
    __device__ __forceinline__ Place(int64_t row, int pitch, int base, int g, int there)
        : at(row * pitch + base + (VEC ? 8 * g : g)), left(there - base - (VEC ? 8 * g : g)) {}
};

// Eight values as loaded: 16-bit ones take four registers until they are used.
// Loads are not of the read-only kind: an output may be the input's buffer.
template <typename T, int LANES, bool VEC>
struct Held;
template <typename T, int LANES>
struct Held<T, LANES, true> {
    static constexpr int kChunks = int(sizeof(T)) / 2;  // of 16 bytes
    uint4 c[kChunks];
    __device__ __forceinline__ void load(const T* p, const Place<LANES, true>& o) {
        const uint4* from = reinterpret_cast<const uint4*>(p + o.at);
#pragma unroll
        for (int h = 0; h < kChunks; ++h) c[h] = o.left > 0 ? __ldcs(from + h) : make_uint4(0, 0, 0, 0);
    }
    // Through shared memory: `to` is the thread's first 16 bytes there, and `step` bytes lie
    // from one to the next.
    __device__ static __forceinline__ void copy(uint32_t to, uint32_t step, const T* p, const Place<LANES, true>& o) {
        const uint4* from = reinterpret_cast<const uint4*>(p + o.at);
        if (o.left > 0)
#pragma unroll
            for (int h = 0; h < kChunks; ++h)  // through the L1: the two of fp32 share sectors
                asm volatile("cp.async.ca.shared.global [%0], [%1], 16;\n" ::"r"(to + h * step), "l"(from + h) : "memory");
    }
    __device__ __forceinline__ void take(uint32_t from, uint32_t step, const Place<LANES, true>& o) {
#pragma unroll
        for (int h = 0; h < kChunks; ++h) {
            c[h] = make_uint4(0, 0, 0, 0);
            if (o.left > 0)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                             : "=r"(c[h].x), "=r"(c[h].y), "=r"(c[h].z), "=r"(c[h].w) : "r"(from + h * step) : "memory");
        }
    }
    __device__ __forceinline__ void get(float2 (&v)[4]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v[2 * h] = make_float2(__uint_as_float(c[h].x), __uint_as_float(c[h].y));
                v[2 * h + 1] = make_float2(__uint_as_float(c[h].z), __uint_as_float(c[h].w));
            }
        } else {
            v[0] = unpack2<T>(c[0].x), v[1] = unpack2<T>(c[0].y), v[2] = unpack2<T>(c[0].z), v[3] = unpack2<T>(c[0].w);
        }
    }
};
template <typename T, int LANES>
struct Held<T, LANES, false> {
    T v[8];
    __device__ __forceinline__ void load(const T* p, const Place<LANES, false>& o) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i * LANES < o.left ? p[o.at + i * LANES] : from_float<T>(0.f);
    }
    __device__ __forceinline__ void get(float2 (&f)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = make_float2(to_float(v[2 * i]), to_float(v[2 * i + 1]));
    }
};

// Copies of a thread for itself: what it reads again it has copied, so no barrier is needed.
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(LEFT) : "memory"); }

template <int LANES, bool VEC, typename T>
__device__ __forceinline__ void store_eight(T* p, const Place<LANES, VEC>& o, const float2 (&v)[4]) {
    if constexpr (VEC) {
        uint4* to = reinterpret_cast<uint4*>(p + o.at);
        if (o.left > 0) {
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    to[h] = make_uint4(__float_as_uint(v[2 * h].x), __float_as_uint(v[2 * h].y),
                                       __float_as_uint(v[2 * h + 1].x), __float_as_uint(v[2 * h + 1].y));
            } else {
                *to = make_uint4(pack2<T>(v[0]), pack2<T>(v[1]), pack2<T>(v[2]), pack2<T>(v[3]));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * LANES < o.left) p[o.at + i * LANES] = from_float<T>(i & 1 ? v[i / 2].y : v[i / 2].x);
    }
}

// Parameters: read by every row, so they stay in the caches.  o: of row 0.
template <int LANES, bool VEC>
__device__ __forceinline__ void load_weights(const float* p, const Place<LANES, VEC>& o, float2 (&v)[4]) {
    if constexpr (VEC) {
        const float4* from = reinterpret_cast<const float4*>(p + o.at);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 f = o.left > 0 ? __ldg(from + h) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[2 * h] = make_float2(f.x, f.y), v[2 * h + 1] = make_float2(f.z, f.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = make_float2(2 * i * LANES < o.left ? __ldg(p + o.at + 2 * i * LANES) : 0.f,
                               (2 * i + 1) * LANES < o.left ? __ldg(p + o.at + (2 * i + 1) * LANES) : 0.f);
    }
}

// v with values dropped and the others scaled.  The whole warp calls it, every group
// for a row of its own.  per: blocks of 8 in a row.  What drops is +0.0 whatever it was.
template <int LANES, bool VEC>
__device__ __forceinline__ void drop_eight(float2 (&v)[4], const Dropout& d, const Masker& m, int64_t row, int per,
                                           int base, int g) {
    if (d.threshold == 0) return;
    if (d.threshold == 65536) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = both(0.f);
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
    for (int i = 0; i < 4; ++i) {
        const float2 f = mul2(v[i], both(d.scale));
        v[i] = make_float2(keep[2 * i] ? f.x : 0.f, keep[2 * i + 1] ? f.y : 0.f);
    }
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
