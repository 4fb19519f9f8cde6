// add_rmsnorm.cu - a branch's dropout, the residual's addition and the
// root-mean-square norm of the sum, in one pass.
//
//   h = residual + drop(x),  rms = sqrt(mean_j h_j^2 + eps),  y = gamma * h / rms
//
// y goes out in x's type, in e4m3 with a scale for each 128 columns (quantize.cu), or
// in e2m1 with a power of two for each 32 (quant.cuh).  The sum stays in fp32 registers
// between its statistic and its norm, so y is not of the rounded h.
//
// Bound by HBM where the stream is fp32: x and residual are read once, h and y written
// once (16384 x 4096, bf16 and an fp32 stream, with dropout: 120 us, 6.7 TB/s).  Where it
// is 16-bit the instructions of a value count as well (8 bytes a value plain 88 us, 6.1
// TB/s; 8192 x 4096 to e4m3 46 us, 5.2; 8192 x 2048 to 4 bits 23 us, 4.7: an SM's 16 warps
// take 56% of its issue slots and wait on their own instructions, not on memory), so values
// are added, multiplied and converted in pairs.  A row lies in the registers of a group of
// lanes, of a warp, or of up to 32 warps that meet once, at a barrier of their own.
#include "eight.cuh"
#include "quant.cuh"

namespace rowops {
namespace {

enum Answer { kPlain, kE4m3, kE2m1 };

struct AddNormArgs {
    const void* x;
    const void* residual;  // may be NULL
    const float* gamma;
    void* h;    // may be NULL
    void* out;
    void* scale;
    float* row_rms;  // may be NULL
    Dropout drop;
    int64_t rows;
    int cols;
    float eps;
    Answer answer;
    RowSplit split;
};

// h of eight columns in fp32.
template <typename T, typename R, int LANES, bool VEC>
struct Sum {
    Held<T, LANES, VEC> x;
    Held<R, LANES, VEC> residual;
    __device__ __forceinline__ void load(const AddNormArgs& a, const Place<LANES, VEC>& o) {
        x.load(static_cast<const T*>(a.x), o);
        if (a.residual) residual.load(static_cast<const R*>(a.residual), o);
    }
    __device__ __forceinline__ void get(const AddNormArgs& a, const Masker& m, int64_t row, int base, int g,
                                        float2 (&v)[4]) const {
        x.get(v);
        drop_eight<LANES, VEC>(v, a.drop, m, row, (a.cols + 7) / 8, base, g);
        if (a.residual) {
            float2 r[4];
            residual.get(r);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = add2(v[i], r[i]);
        }
    }
};

// y of eight columns.
template <int LANES, bool VEC>
__device__ __forceinline__ void normed(const AddNormArgs& a, int base, int g, int cols, float inv, const float2 (&h)[4],
                                       float2 (&y)[4]) {
    float2 gamma[4];
    load_weights<LANES, VEC>(a.gamma, Place<LANES, VEC>(0, 0, base, g, cols), gamma);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mul2(mul2(h[i], both(inv)), gamma[i]);
}

// Eight columns of the answer.
template <typename T, int LANES, bool VEC>
__device__ __forceinline__ void answer_eight(const AddNormArgs& a, int64_t row, int base, int g, int cols,
                                             const float2 (&y)[4]) {
    if (a.answer == kPlain) {
        store_eight<LANES, VEC>(static_cast<T*>(a.out), Place<LANES, VEC>(row, a.cols, base, g, cols), y);
        return;
    }
    if (a.answer == kE4m3) {
        store_e4m3<LANES, VEC>(static_cast<uint8_t*>(a.out) + row * a.cols,
                               static_cast<float*>(a.scale) + row * ((a.cols + 127) / 128), base, g, cols, y);
    } else {
        store_mx4<LANES, VEC>(static_cast<uint8_t*>(a.out) + row * ((a.cols + 1) / 2),
                              static_cast<uint8_t*>(a.scale) + row * ((a.cols + 31) / 32), base, g, cols, y);
    }
}

template <typename T, typename R, int LANES, int NV, bool VEC, int MOST>
__global__ void __launch_bounds__(MOST) add_rmsnorm_rows(const AddNormArgs a) {
    __shared__ float scratch[2][32];
    let_next_start();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot = warp / a.split.warps, w = warp % a.split.warps, g = lane % LANES;
    constexpr int kGroups = 32 / LANES;
    const float inv_cols = 1.0f / float(a.cols);
    const Masker masker(a.drop);
    int turn = 0;
    for (int64_t first = (int64_t(blockIdx.x) * a.split.slots + slot) * kGroups; first < a.rows;
         first += int64_t(gridDim.x) * a.split.slots * kGroups, turn ^= 1) {
        const int64_t row = first + lane / LANES;
        const int cols = row < a.rows ? a.cols : 0;
        Sum<T, R, LANES, VEC> in[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k)
            in[k].load(a, Place<LANES, VEC>(row, a.cols, (k * a.split.warps + w) * 256, g, cols));
        float2 h[NV][4], squares = both(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int base = (k * a.split.warps + w) * 256;
            in[k].get(a, masker, row, base, g, h[k]);
#pragma unroll
            for (int i = 0; i < 4; ++i) squares = fma2(h[k][i], h[k][i], squares);  // 0 past the row's end
            if (a.h) store_eight<LANES, VEC>(static_cast<R*>(a.h), Place<LANES, VEC>(row, a.cols, base, g, cols), h[k]);
        }
        const float sum = sum_of_row<LANES>(squares.x + squares.y, scratch[turn], a.split.warps, slot, w);
        const float rms = sqrtf(sum * inv_cols + a.eps);
        if (a.row_rms && w == 0 && g == 0 && row < a.rows) a.row_rms[row] = rms;
        const float inv = 1.0f / rms;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int base = (k * a.split.warps + w) * 256;
            float2 y[4];
            normed<LANES, VEC>(a, base, g, cols, inv, h[k], y);
            answer_eight<T, LANES, VEC>(a, row, base, g, cols, y);
        }
    }
}

// Many rows on 16-byte boundaries: a block stays on its SM, with gamma in registers, and
// each thread has the next rows of its own columns copied to places in shared memory.
// A lane holds 8 columns of rows up to 1024 values and two blocks share an SM; longer rows
// take 16, in one block with twice the registers.
constexpr int kStages = 2;
template <int NV>
constexpr int kBlocks = NV == 1 ? 2 : 1;
template <typename T, typename R>
constexpr int kPlaces = Held<T, 32, true>::kChunks + Held<R, 32, true>::kChunks;  // of 16 bytes, a row

template <typename T, typename R, int LANES, int NV>
__global__ void __launch_bounds__(512, kBlocks<NV>) add_rmsnorm_stream(const AddNormArgs a) {
    extern __shared__ __align__(16) unsigned char shared[];
    __shared__ float scratch[2][32];
    let_next_start();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot = warp / a.split.warps, w = warp % a.split.warps, g = lane % LANES;
    constexpr int kGroups = 32 / LANES;
    const float inv_cols = 1.0f / float(a.cols);
    const Masker masker(a.drop);
    const auto base_of = [&](int k) { return (k * a.split.warps + w) * 256; };
    float2 gamma[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k)
        load_weights<LANES, true>(a.gamma, Place<LANES, true>(0, 0, base_of(k), g, a.cols), gamma[k]);
    using HeldT = Held<T, LANES, true>;
    using HeldR = Held<R, LANES, true>;
    const uint32_t step = blockDim.x * 16;  // from place to place
    const uint32_t places = uint32_t(__cvta_generic_to_shared(shared)) + threadIdx.x * 16;
    const int64_t first = (int64_t(blockIdx.x) * a.split.slots + slot) * kGroups;
    const int64_t stride = int64_t(gridDim.x) * a.split.slots * kGroups;
    const auto begin = [&](int64_t from, uint32_t at) {  // copies of the rows at `from`
        const int64_t row = from + lane / LANES;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const Place<LANES, true> o(row, a.cols, base_of(k), g, row < a.rows ? a.cols : 0);
            HeldT::copy(at, step, static_cast<const T*>(a.x), o);
            at += HeldT::kChunks * step;
            if (a.residual) HeldR::copy(at, step, static_cast<const R*>(a.residual), o);
            at += HeldR::kChunks * step;
        }
        copies_end();
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) begin(first + s * stride, places + s * NV * kPlaces<T, R> * step);
    int turn = 0;
    for (int64_t from = first; from < a.rows; from += stride, turn ^= 1) {
        const int64_t row = from + lane / LANES;
        const int there = row < a.rows ? a.cols : 0;
        const uint32_t stage = places + turn * NV * kPlaces<T, R> * step;  // kStages is 2
        float2 h[NV][4], squares = both(0.f);
        copies_wait<kStages - 1>();
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const Place<LANES, true> o(row, a.cols, base_of(k), g, there);
            const uint32_t at = stage + k * kPlaces<T, R> * step;
            Sum<T, R, LANES, true> in;
            in.x.take(at, step, o);
            if (a.residual) in.residual.take(at + HeldT::kChunks * step, step, o);
            in.get(a, masker, row, base_of(k), g, h[k]);
#pragma unroll
            for (int i = 0; i < 4; ++i) squares = fma2(h[k][i], h[k][i], squares);
            if (a.h) store_eight<LANES, true>(static_cast<R*>(a.h), o, h[k]);
        }
        begin(from + kStages * stride, stage);  // where all has been read
        const float sum = sum_of_row<LANES>(squares.x + squares.y, scratch[turn], a.split.warps, slot, w);
        const float rms = sqrtf(sum * inv_cols + a.eps);
        if (a.row_rms && w == 0 && g == 0 && row < a.rows) a.row_rms[row] = rms;
        const float2 inv = both(1.0f / rms);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) h[k][i] = mul2(mul2(h[k][i], inv), gamma[k][i]);
            answer_eight<T, LANES, true>(a, row, base_of(k), g, there, h[k]);
        }
    }
}

// Rows of more than 16384 values: one block a row, which reads x and the residual a
// second time, from the L2, for the answer.  h is written only then: it may lie where
// the residual does.
template <typename T, typename R, bool VEC>
__global__ void __launch_bounds__(1024) add_rmsnorm_long(const AddNormArgs a) {
    __shared__ float scratch[2][32];
    let_next_start();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float inv_cols = 1.0f / float(a.cols);
    const Masker masker(a.drop);
    const int64_t units = (int64_t(a.cols) + 255) / 256;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        float2 squares = both(0.f);
#pragma unroll VEC ? 2 : 1
        for (int64_t u = w; u < units; u += 32) {
            Sum<T, R, 32, VEC> in;
            float2 h[4];
            in.load(a, Place<32, VEC>(row, a.cols, int(u * 256), lane, a.cols));
            in.get(a, masker, row, int(u * 256), lane, h);
#pragma unroll
            for (int i = 0; i < 4; ++i) squares = fma2(h[i], h[i], squares);
        }
        const float rms = sqrtf(sum_of_row<32>(squares.x + squares.y, scratch[turn], 32, 0, w) * inv_cols + a.eps);
        if (a.row_rms && threadIdx.x == 0) a.row_rms[row] = rms;
        const float inv = 1.0f / rms;
#pragma unroll VEC ? 2 : 1
        for (int64_t u = w; u < units; u += 32) {
            const int base = int(u * 256);
            const Place<32, VEC> o(row, a.cols, base, lane, a.cols);
            Sum<T, R, 32, VEC> in;
            float2 h[4], y[4];
            in.load(a, o);
            in.get(a, masker, row, base, lane, h);
            if (a.h) store_eight<32, VEC>(static_cast<R*>(a.h), o, h);
            normed<32, VEC>(a, base, lane, a.cols, inv, h, y);
            answer_eight<T, 32, VEC>(a, row, base, lane, a.cols, y);
        }
    }
}

}  // namespace

cudaError_t launch_add_rmsnorm_fwd(const void* x, const void* residual, const float* gamma, const uint64_t* rng,
                                   void* h, void* out, void* scale, float* row_rms, int64_t rows, int64_t cols,
                                   float eps, float p, int x_type, int h_type, int out_type, cudaStream_t stream) {
    AddNormArgs a{x, residual, gamma, h, out, scale, row_rms, dropout_of(rng, p), rows, int(cols), eps, kPlain, {1, 1}};
    if (out_type == ROWOPS_E4M3) a.answer = kE4m3;
    if (out_type == ROWOPS_E2M1) a.answer = kE2m1;
    const bool vec = cols % 8 == 0 && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) |
                                        reinterpret_cast<uintptr_t>(gamma) | reinterpret_cast<uintptr_t>(h) |
                                        reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    const int units = int((cols + 255) / 256);
    const int64_t sms = sm_count() > 0 ? sm_count() : 132;
    cudaError_t e = cudaSuccess;
    auto go = [&](auto kernel, int groups, int warps, int slots) {
        a.split = {warps, slots};
        const int64_t per = int64_t(slots) * groups, blocks = (rows + per - 1) / per, most = int64_t(1) << 20;
        kernel<<<unsigned(blocks < most ? blocks : most), unsigned(warps * slots * 32), 0, stream>>>(a);
    };
    with_branch_types(x_type, h_type, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        // Rows through shared memory against rows straight to registers: short rows (16384 x 768
        // bf16: 19.0 and 22.4 us; 65536 x 256: 24.5 and 43), and 16-bit streams whose rows take
        // the quantiser's or the generator's work (8192 x 2048 to 4 bits: 23.0 and 26.5; 16384 x
        // 4096 with dropout: 88 and 101), not plain wide ones (16384 x 4096: 92 and 88; fp32 stream
        // with dropout: 132 to 146, and 120).
        const bool busy = sizeof(R) == 2 && (a.answer != kPlain || a.drop.threshold != 0);
        if (vec && rows > 4 * sms && (units <= 4 || (units <= 32 && busy))) {
            const int nv = units > 4 ? 2 : 1, warps = (units + nv - 1) / nv;
            a.split = {warps, 16 / warps};
            auto stream_rows = [&](auto kernel, int groups, int64_t most) {
                const int threads = a.split.warps * a.split.slots * 32;
                const size_t smem = size_t(kStages) * nv * kPlaces<T, R> * 16 * threads;
                const int64_t per = int64_t(a.split.slots) * groups, blocks = (rows + per - 1) / per;
                if (smem > 47 * 1024) e = allow_smem(kernel, smem);  // 48 KB with the static part need no leave
                if (e == cudaSuccess) kernel<<<unsigned(blocks < most ? blocks : most), unsigned(threads), smem, stream>>>(a);
            };
            if (cols <= 64) stream_rows(add_rmsnorm_stream<T, R, 8, 1>, 4, sms * kBlocks<1>);
            else if (cols <= 128) stream_rows(add_rmsnorm_stream<T, R, 16, 1>, 2, sms * kBlocks<1>);
            else if (nv == 1) stream_rows(add_rmsnorm_stream<T, R, 32, 1>, 1, sms * kBlocks<1>);
            else stream_rows(add_rmsnorm_stream<T, R, 32, 2>, 1, sms * kBlocks<2>);
            return;
        }
        auto pick = [&](auto v) {
            constexpr bool VEC = decltype(v)::value;
            if (VEC && cols <= 64) go(add_rmsnorm_rows<T, R, VEC ? 8 : 32, 1, VEC, 128>, 4, 1, 4);
            else if (VEC && cols <= 128) go(add_rmsnorm_rows<T, R, VEC ? 16 : 32, 1, VEC, 128>, 2, 1, 4);
            else if (units == 1) go(add_rmsnorm_rows<T, R, 32, 1, VEC, 128>, 1, 1, 4);
            else if (units <= 32 && rows <= 4 * sms)
                go(add_rmsnorm_rows<T, R, 32, 1, VEC, 1024>, 1, units, units <= 4 ? 2 : 1);
            else if (units <= 64) {
                const int warps = (units + 1) / 2;
                go(add_rmsnorm_rows<T, R, 32, 2, VEC, 1024>, 1, warps, warps <= 4 ? 8 / warps : 1);
            } else
                go(add_rmsnorm_long<T, R, VEC>, 1, 32, 1);
        };
        if (vec) pick(std::true_type{});
        else pick(std::false_type{});
    });
    if (e != cudaSuccess) return e;
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace rowops
