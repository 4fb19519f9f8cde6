// quantize_mx4.cu - microscaled 4-bit values (e2m1) with a power of two for each
// block of 32 columns of a row (quant.cuh).
//
// Bound by HBM: reads the input once, writes 17 bytes for 32 values.  Four lanes hold
// a block.  Where rows are whole blocks the matrix is one run of chunks of eight values,
// of which a thread has four on their way (16384 x 4096 bf16: 27 us, 6.2 TB/s; one at a
// time 49, eight 36), and the maximum of 16-bit values is taken on their bits, two at a
// time.  Other rows are a run of chunks too, with the last block's filled up to four
// (16384 x 1000: 10.3 us with four on their way, 12.8 with one); chunks that start anywhere
// come by words and go by bytes (x 1001: 16.9 us with two, 17.9 with one, 18.4 with four).
#include "bytes.cuh"
#include "eight.cuh"
#include "quant.cuh"

namespace rowops {
namespace {

// The largest magnitude of eight values as fp32 bits; 16-bit values are compared as they
// are, two at a time.
template <typename T>
__device__ __forceinline__ uint32_t most_of(const Held<T, 32, true>& x) {
    if constexpr (sizeof(T) == 4) {
        uint32_t m = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            m = max(max(m, max(x.c[h].x & 0x7fffffffu, x.c[h].y & 0x7fffffffu)),
                    max(x.c[h].z & 0x7fffffffu, x.c[h].w & 0x7fffffffu));
        return group_max_bits<4>(m);
    } else {
        const uint4 w = x.c[0];
        uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                              __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
#pragma unroll
        for (int o = 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(kFullMask, m, o));
        return __float_as_uint(unpack2<T>(max(m & 0xffffu, m >> 16)).x);
    }
}

// Rows that are whole blocks: the matrix as one run of chunks of eight values, ITEMS of
// them a thread.
template <typename T, int ITEMS, int THREADS>
__global__ void __launch_bounds__(THREADS)
    quantize_mx4_run(const T* x, uint32_t* __restrict__ q, uint8_t* __restrict__ scale, int64_t chunks) {
    let_next_start();
    const int64_t first = int64_t(blockIdx.x) * (THREADS * ITEMS) + threadIdx.x;
    Held<T, 32, true> in[ITEMS];
#pragma unroll
    for (int n = 0; n < ITEMS; ++n)
        in[n].load(x, Place<32, true>(first + n * THREADS, 8, 0, 0, first + n * THREADS < chunks ? 8 : 0));
#pragma unroll
    for (int n = 0; n < ITEMS; ++n) {
        const int64_t at = first + n * THREADS;
        const uint32_t code = mx4_code(most_of<T>(in[n]));
        float2 v[4];
        in[n].get(v);
        if (at < chunks) {
            q[at] = mx4_eight(v, code);
            if ((threadIdx.x & 3) == 0) scale[at / 4] = uint8_t(code);
        }
    }
}

struct Mx4Args {
    const void* x;
    uint8_t* q;
    uint8_t* scale;
    int64_t rows;
    int cols;
    Divisor32 across;  // chunks of a row, filled up to whole blocks of four
};

// Eight values that start anywhere, of which the first `left` are there.
template <typename T>
__device__ __forceinline__ void load_anywhere(Held<T, 32, true>& x, const T* from, int left, const T* begin, const T* end) {
    if constexpr (sizeof(T) == 4) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = i < left ? __float_as_uint(__ldcs(reinterpret_cast<const float*>(from) + i)) : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) x.c[h] = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
    } else {
        const uint8_t* at = reinterpret_cast<const uint8_t*>(from);
        const int off = int(reinterpret_cast<uintptr_t>(at) & 2);
        uint32_t w[5];
        words_at(at - off, reinterpret_cast<const uint8_t*>(begin), reinterpret_cast<const uint8_t*>(end), w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = __funnelshift_r(w[i], w[i + 1], 8 * off);
            if (2 * i + 1 >= left) w[i] &= 2 * i < left ? 0xffffu : 0u;  // the next row's
        }
        x.c[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Other rows: chunks of eight columns, filled up to whole blocks in every row, ITEMS a
// thread.  VEC: rows are whole chunks on 16-byte boundaries; others start anywhere.
template <typename T, bool VEC, int ITEMS, int THREADS>
__global__ void __launch_bounds__(THREADS) quantize_mx4_rows(const Mx4Args a) {
    let_next_start();
    const T* x = static_cast<const T*>(a.x);
    const int64_t block = int64_t(blockIdx.x) * (THREADS * ITEMS);
    const int64_t row0 = block <= UINT32_MAX ? int64_t(uint32_t(block) / a.across.d) : block / a.across.d;
    const uint32_t in_row = uint32_t(block - row0 * a.across.d) + threadIdx.x;
    // the n-th chunk's row, its place there and how many of its values there are
    const auto place = [&](int n, int64_t& row, int& chunk) {
        const uint32_t at = in_row + n * THREADS, down = a.across.quotient(at);
        row = row0 + down;
        chunk = int(at - down * a.across.d);
        return row < a.rows ? min(a.cols - 8 * chunk, 8) : 0;
    };
    Held<T, 32, true> in[ITEMS];
#pragma unroll
    for (int n = 0; n < ITEMS; ++n) {
        int64_t row;
        int chunk;
        const int left = place(n, row, chunk);
        if constexpr (VEC) {
            in[n].load(x, Place<32, true>(row, a.cols, 8 * chunk, 0, left > 0 ? a.cols : 0));
        } else {
#pragma unroll
            for (auto& c : in[n].c) c = make_uint4(0, 0, 0, 0);
            if (left > 0) load_anywhere(in[n], x + row * a.cols + 8 * chunk, left, x, x + a.rows * a.cols);
        }
    }
#pragma unroll
    for (int n = 0; n < ITEMS; ++n) {
        const uint32_t code = mx4_code(most_of<T>(in[n]));
        float2 v[4];
        in[n].get(v);
        const uint32_t q = mx4_eight(v, code);
        int64_t row;
        int chunk;
        const int left = place(n, row, chunk);
        if (left > 0) {
            uint8_t* to = a.q + row * ((a.cols + 1) / 2) + 4 * chunk;
            if constexpr (VEC) {
                *reinterpret_cast<uint32_t*>(to) = q;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (2 * i < left) to[i] = uint8_t(q >> (8 * i));
            }
            if (chunk % 4 == 0) a.scale[row * ((a.cols + 31) / 32) + chunk / 4] = uint8_t(code);
        }
    }
}

}  // namespace

cudaError_t launch_quantize_mx4(const void* x, uint8_t* q, uint8_t* scale, int64_t rows, int64_t cols, int x_type,
                                cudaStream_t stream) {
    const bool vec = cols % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 && reinterpret_cast<uintptr_t>(q) % 4 == 0;
    const bool run = vec && cols % 32 == 0;
    const int64_t across = run ? cols / 8 : (cols + 31) / 32 * 4, chunks = rows * across;
    const Mx4Args a{x, q, scale, rows, int(cols), Divisor32(uint32_t(across))};
    // A chunk a thread as long as the SMs hold all of them at once (bf16, one and more: 64 x 4096 1.5 and
    // 1.9 us, 512 x 4096 2.7 and 2.6, 1024 x 4096 5.0 and 3.8; 64 x 4088 1.9 and 2.2, 1024 x 4088 5.0
    // and 4.3; 64 x 4001 1.9 and 2.4, 512 x 4001 3.6 and 3.8, 2048 x 4001 10.1 and 9.6).
    const bool few = chunks < 2048 * int64_t(sm_count());
    auto grid = [&](int per) { return unsigned((chunks + per - 1) / per); };
    with_type(x_type, [&](auto t) {
        using T = decltype(t);
        const T* from = static_cast<const T*>(x);
        uint32_t* words = reinterpret_cast<uint32_t*>(q);
        if (run && few) quantize_mx4_run<T, 1, 128><<<grid(128), 128, 0, stream>>>(from, words, scale, chunks);
        else if (run) quantize_mx4_run<T, 4, 256><<<grid(4 * 256), 256, 0, stream>>>(from, words, scale, chunks);
        else if (vec && few) quantize_mx4_rows<T, true, 1, 128><<<grid(128), 128, 0, stream>>>(a);
        else if (vec) quantize_mx4_rows<T, true, 4, 256><<<grid(4 * 256), 256, 0, stream>>>(a);
        else if (few) quantize_mx4_rows<T, false, 1, 128><<<grid(128), 128, 0, stream>>>(a);
        else quantize_mx4_rows<T, false, 2, 256><<<grid(2 * 256), 256, 0, stream>>>(a);
    });
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace rowops
