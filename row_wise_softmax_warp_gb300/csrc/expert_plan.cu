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
// kOneBlockPairs pairs are one launch.  262144 x 2 pairs of 64 experts: 15 us.
#include "groups.cuh"
#include "launch.h"

namespace rowops {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kOneBlockPairs = 4096;

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
__global__ void __launch_bounds__(kPlanThreads) plan_count(const float* indices, const float* values,
                                                           int32_t* counts, int pairs, int experts, int run) {
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < experts; e += kPlanThreads) hist[e] = 0;
    __syncthreads();
    int begin, end;
    my_run(pairs, run, begin, end);
    for (int p = begin + threadIdx.x; p < end; p += kPlanThreads) {
        const int e = pair_expert(indices, values, p, experts);
        if (e < experts) atomicAdd(&hist[e], 1);  // integer counts: the order of the adds does not matter
    }
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += kPlanThreads)
        counts[int64_t(blockIdx.x) * experts + e] = hist[e];
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}

// Shared memory: total[experts] (all blocks), mine[experts] (blocks before this
// one), at[kPlanWarps][experts] (each warp's next slot per expert).
__global__ void __launch_bounds__(kPlanThreads)
    plan_place(const float* indices, const float* values, const int32_t* counts, int32_t* offsets, int32_t* order,
               int32_t* slot, int pairs, int experts, int run) {
    extern __shared__ int sh[];
    int* total = sh;
    int* mine = sh + experts;
    int* at = sh + 2 * experts;
    __shared__ int warp_sum[kPlanWarps];
    __shared__ int all;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = gridDim.x, me = blockIdx.x;

    int begin, end;
    my_run(pairs, run, begin, end);
    const int per = ((end - begin) + kPlanWarps - 1) / kPlanWarps;
    const int wb = min(begin + warp * per, end), we = min(wb + per, end);

    for (int i = tid; i < experts * kPlanWarps; i += kPlanThreads) at[i] = 0;
    __syncthreads();
    for (int p = wb + lane; p < we; p += 32) {
        const int e = pair_expert(indices, values, p, experts);
        if (e < experts) atomicAdd(&at[warp * experts + e], 1);
    }
    __syncthreads();
    for (int e = tid; e < experts; e += kPlanThreads) {
        int sum = 0;
        if (blocks == 1)
            for (int w = 0; w < kPlanWarps; ++w) sum += at[w * experts + e];
        total[e] = sum;
        mine[e] = 0;
    }
    __syncthreads();
    if (blocks > 1) {
        asm volatile("griddepcontrol.wait;\n" ::: "memory");  // plan_count's writes
        // `parts` threads per expert add up every parts-th block's counts
        const int parts = max(1, kPlanThreads / experts);
        for (int i = tid; i < experts * parts; i += kPlanThreads) {
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
    // exclusive scan of total over the experts (at most 1024: two per thread)
    constexpr int kPer = kMaxExperts / kPlanThreads;
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
    if (tid == kPlanThreads - 1) all = base;
    __syncthreads();
    if (me == 0 && tid == 0) offsets[experts] = all;
    // each warp's first slot per expert: this block's, then the warps before it
    for (int e = tid; e < experts; e += kPlanThreads) {
        int next = mine[e];
        for (int w = 0; w < kPlanWarps; ++w) {
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
    for (int64_t s = all + int64_t(me) * kPlanThreads + tid; s < pairs; s += int64_t(blocks) * kPlanThreads)
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
    const size_t smem = size_t(ne) * 4 * (2 + kPlanWarps);
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(plan_place, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
    }
    int32_t* counts = static_cast<int32_t*>(workspace);
    if (blocks > 1) {
        plan_count<<<blocks, kPlanThreads, size_t(ne) * 4, stream>>>(indices, values, counts, int(pairs), ne, run);
        note_launches(1);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 1 : 0;  // alone it must wait for whatever ran before
    const cudaError_t e = cudaLaunchKernelEx(&cfg, plan_place, indices, values, static_cast<const int32_t*>(counts),
                                             offsets, order, slot, int(pairs), ne, run);
    note_launches(1);
    return e;
}

}  // namespace rowops
