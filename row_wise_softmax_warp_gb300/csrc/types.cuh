// types.cuh - the element types of the expert operators (fp32, fp16, bf16) and
// chunked loads and stores that compute in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "launch.h"
#include "rowops.h"

namespace rowops {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// A chunk of V values is moved by one access of V * sizeof(T) bytes (2..16).
template <int BYTES>
struct RawOf;
template <>
struct RawOf<2> { using type = unsigned short; };
template <>
struct RawOf<4> { using type = unsigned int; };
template <>
struct RawOf<8> { using type = uint2; };
template <>
struct RawOf<16> { using type = uint4; };

template <typename T, int V>
struct Chunk {
    using Raw = typename RawOf<V * int(sizeof(T))>::type;
    union {
        Raw raw;
        T v[V];
    };
    __device__ __forceinline__ Chunk() : raw() {}
    __device__ __forceinline__ void load(const T* p) { raw = __ldg(reinterpret_cast<const Raw*>(p)); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Raw*>(p) = raw; }
    // for what is touched once: the lines leave the caches first
    __device__ __forceinline__ void load_once(const T* p) { raw = __ldcs(reinterpret_cast<const Raw*>(p)); }
    __device__ __forceinline__ void store_once(T* p) const { __stcs(reinterpret_cast<Raw*>(p), raw); }
    __device__ __forceinline__ float get(int i) const { return to_float(v[i]); }
    __device__ __forceinline__ void set(int i, float f) { v[i] = from_float<T>(f); }
};

// Values per chunk of a kernel that reads A and writes B: 16 bytes of the wider.
template <typename A, typename B>
constexpr int chunk_of() {
    return 16 / int(sizeof(A) > sizeof(B) ? sizeof(A) : sizeof(B));
}

// Host: f(T{}) with the element type of a rowops_dtype; false for another value.
template <typename F>
bool with_type(int dtype, F&& f) {
    switch (dtype) {
        case ROWOPS_F32: f(float{}); return true;
        case ROWOPS_F16: f(__half{}); return true;
        case ROWOPS_BF16: f(__nv_bfloat16{}); return true;
        default: return false;
    }
}

}  // namespace rowops
