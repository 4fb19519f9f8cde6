// expert_plan.cu - (token, choice) pairs grouped by expert: a stable counting
// sort by expert number.
//
//   c_e = #{pairs of expert e},  offsets_e = sum_{e' < e} c_e',
//   slot_p = offsets_e + #{p' < p of the same expert e},  order[slot_p] = p.
//
// What bounds it: 16 bytes a pair (index, value, order, slot); below about a
// million pairs the launches.  Each block owns a contiguous run of pairs and
// each of its warps a contiguous run of those, so ranks follow from counts
// alone and no atomic's order reaches the result.  plan_count writes each
// block's counts; plan_place, a programmatic dependent that counts its own pairs
// meanwhile, adds up the counts of the blocks before it (read from the L2, the
// blocks split among threads: one thread an expert took 8 of 21 us), ranks its
// pairs and writes them.  One block needs no counts from others: up to
// kOneBlockPairs pairs are one launch.  262144 x 2 pairs of 64 experts: 14.7 us, of which
// 2 are the trip to memory for a value that starts only after its index has come back
// (12.2 without values; 12.9 in a trial that loads both at once).
#include "groups.cuh"
#include "launch.h"

namespace rowops {
namespace {

// One block alone is faster with 512 threads (64 pairs: 2.8 against 3.5 us), many
// with 1024 (524288 pairs of 256 experts: 17.9 against 23.0 us).  2048 pairs: 5.6 us
// in one block, 6.4 in two launches; 4096 pairs: 8.9 and 6.4.
constexpr int kOneThreads = 512, kManyThreads = 1024;
constexpr int kOneBlockPairs = 2048;

// Expert of pair p, or `experts` for a pair that is left out.
__device__ __forceinline__ int pair_expert(const float* indices, const float* values, int p, int experts) {
    const float i = __ldg(indices + p);
    const bool there = i >= 0.0f && i < float(experts) && (values == nullptr || __ldg(values + p) != 0.0f);
    return there ? int(i) : experts;
}

__device__ __forceinline__ void my_run(int pairs, int run, int& begin, int& end) {
    const int64_t b = int64_t(blockIdx.x) * run;
    begin = int(b < pairs ? b : pairs);
    end = int(b + run < pairs ? b + run : pairs);
}

// counts[block][e]
__global__ void __launch_bounds__(kManyThreads) plan_count(const float* indices, const float* values,
                                                           int32_t* counts, int pairs, int experts, int run) {
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < experts; e += kManyThreads) hist[e] = 0;
    __syncthreads();
    int begin, end;
    my_run(pairs, run, begin, end);
    for (int p = begin + threadIdx.x; p < end; p += kManyThreads) {
        const int e = pair_expert(indices, values, p, experts);
        if (e < experts) atomicAdd(&hist[e], 1);  // integer counts: the order of the adds does not matter
    }
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += kManyThreads)
        counts[int64_t(blockIdx.x) * experts + e] = hist[e];
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}

// Shared memory: total[experts] (all blocks), mine[experts] (blocks before this
// one), at[warps][experts] (each warp's next slot per expert).
template <int NT>
__global__ void __launch_bounds__(NT)
    plan_place(const float* indices, const float* values, const int32_t* counts, int32_t* offsets, int32_t* order,
               int32_t* slot, int pairs, int experts, int run) {
    constexpr int kWarps = NT / 32;
    extern __shared__ int sh[];
    int* total = sh;
    int* mine = sh + experts;
    int* at = sh + 2 * experts;
    __shared__ int warp_sum[kWarps];
    __shared__ int all;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = gridDim.x, me = blockIdx.x;

    int begin, end;
    my_run(pairs, run, begin, end);
    const int per = ((end - begin) + kWarps - 1) / kWarps;
    const int wb = min(begin + warp * per, end), we = min(wb + per, end);

    for (int i = tid; i < experts * kWarps; i += NT) at[i] = 0;
    __syncthreads();
    for (int p = wb + lane; p < we; p += 32) {
        const int e = pair_expert(indices, values, p, experts);
        if (e < experts) atomicAdd(&at[warp * experts + e], 1);
    }
    __syncthreads();
    for (int e = tid; e < experts; e += NT) {
        int sum = 0;
        if (blocks == 1)
            for (int w = 0; w < kWarps; ++w) sum += at[w * experts + e];
        total[e] = sum;
        mine[e] = 0;
    }
    __syncthreads();
    if (blocks > 1) {
        asm volatile("griddepcontrol.wait;\n" ::: "memory");  // plan_count's writes
        // `parts` threads per expert add up every parts-th block's counts
        const int parts = max(1, NT / experts);
        for (int i = tid; i < experts * parts; i += NT) {
            const int e = i % experts;
            int before = 0, sum = 0;
#pragma unroll 8
            for (int b = i / experts; b < blocks; b += parts) {
                const int c = __ldcg(counts + int64_t(b) * experts + e);
                before += b < me ? c : 0;
                sum += c;
            }
            atomicAdd(&total[e], sum);
            atomicAdd(&mine[e], before);
        }
        __syncthreads();
    }
    // exclusive scan of total over the experts
    constexpr int kPer = kMaxExperts / NT;
    int v[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = tid * kPer + i;
        v[i] = e < experts ? total[e] : 0;
        sum += v[i];
    }
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFullMask, upto, o);
        if (lane >= o) upto += u;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    int base = upto - sum;
    for (int w = 0; w < warp; ++w) base += warp_sum[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = tid * kPer + i;
        if (e < experts) {
            if (me == 0) offsets[e] = base;
            mine[e] += base;
        }
        base += v[i];
    }
    if (tid == NT - 1) all = base;
    __syncthreads();
    if (me == 0 && tid == 0) offsets[experts] = all;
    // each warp's first slot per expert: this block's, then the warps before it
    for (int e = tid; e < experts; e += NT) {
        int next = mine[e];
        for (int w = 0; w < kWarps; ++w) {
            const int c = at[w * experts + e];
            at[w * experts + e] = next;
            next += c;
        }
    }
    __syncthreads();
    int* next = at + warp * experts;
    for (int p0 = wb; p0 < we; p0 += 32) {
        const int p = p0 + lane;
        const int e = p < we ? pair_expert(indices, values, p, experts) : experts;
        const unsigned same = __match_any_sync(kFullMask, e);
        const unsigned before = same & ((1u << lane) - 1u);
        int s = -1;
        if (e < experts) s = next[e] + __popc(before);
        __syncwarp();
        if (e < experts && before == 0) next[e] += __popc(same);
        __syncwarp();
        if (p < we) {
            slot[p] = s;
            if (s >= 0) order[s] = p;
        }
    }
    // the slots past the last pair
    for (int64_t s = all + int64_t(me) * NT + tid; s < pairs; s += int64_t(blocks) * NT)
        order[s] = -1;
}

// Blocks and pairs per block: runs of at least 1024 pairs, at most one block per SM.
void plan_shape(int64_t pairs, int& blocks, int& run) {
    if (pairs <= kOneBlockPairs) {
        blocks = 1;
        run = int(pairs);
        return;
    }
    const int sms = sm_count() > 0 ? sm_count() : 1;
    int64_t b = (pairs + 1023) / 1024;
    if (b > sms) b = sms;
    blocks = int(b);
    run = int((pairs + b - 1) / b);
}

}  // namespace

size_t expert_plan_workspace(int64_t pairs, int64_t experts) {
    int blocks, run;
    plan_shape(pairs, blocks, run);
    return blocks > 1 ? size_t(blocks) * size_t(experts) * 4 : 0;
}

cudaError_t launch_expert_plan(const float* indices, const float* values, int32_t* offsets, int32_t* order,
                               int32_t* slot, int64_t pairs, int64_t experts, void* workspace, cudaStream_t stream) {
    int blocks, run;
    plan_shape(pairs, blocks, run);
    const int ne = int(experts);
    const auto place = blocks > 1 ? plan_place<kManyThreads> : plan_place<kOneThreads>;
    const int threads = blocks > 1 ? kManyThreads : kOneThreads;
    const size_t smem = size_t(ne) * 4 * (2 + threads / 32);
    if (smem > 48 * 1024) {
        const cudaError_t e = allow_smem(place, smem);
        if (e != cudaSuccess) return e;
    }
    int32_t* counts = static_cast<int32_t*>(workspace);
    if (blocks > 1) {
        plan_count<<<blocks, kManyThreads, size_t(ne) * 4, stream>>>(indices, values, counts, int(pairs), ne, run);
        note_launches(1);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 1 : 0;  // alone it must wait for whatever ran before
    const cudaError_t e = cudaLaunchKernelEx(&cfg, place, indices, values, static_cast<const int32_t*>(counts),
                                             offsets, order, slot, int(pairs), ne, run);
    note_launches(1);
    return e;
}

}  // namespace rowops
