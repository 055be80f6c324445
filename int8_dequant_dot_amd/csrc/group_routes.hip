// group_routes.hip -- routes in the order of their experts (a stable counting
// sort), for products that take each expert's rows together.
//
//     route p = token * routes + i leads to expert ids[p]; routes of one expert
//     keep their order.  slots[p]: its place; rows[place]: its token;
//     offsets[e]: the first place of expert e.
//
// A route whose id is no expert has slot -1, and rows past the last place are -1.
//
// Launches bound it: one for up to 2048 routes (5 us), two for more.  524288 routes of 256
// experts take 14.8 us, where their 6.3 MB would take 1.4; a table of counts added through
// LDS atomics took 25.
#include "device_common.hpp"
#include "internal.hpp"

namespace loom {

namespace {

// Lanes of this wave that hold the same key, for keys below 2^bits.
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot(key >> b & 1);
        same &= (key >> b & 1) ? set : ~set;
    }
    return same;
}

__device__ __forceinline__ int expert_of(const GroupArgs &a, int64_t p, int64_t end) {
    const int id = p < end ? a.ids[p] : -1;
    return id >= 0 && id < a.experts ? id : a.experts;  // the last key: none
}

// Routes of each expert in this block's part -> counts[block][expert].
__global__ __launch_bounds__(kGroupWaves * kWave) void group_count_kernel(GroupArgs a) {
    __shared__ int count[kGroupMaxExperts + 1];
    for (int e = threadIdx.x; e <= a.experts; e += blockDim.x) count[e] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * a.part, end = begin + a.part < a.pairs ? begin + a.part : a.pairs;
    for (int64_t p = begin + threadIdx.x; p < end; p += blockDim.x) atomicAdd(&count[expert_of(a, p, end)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) a.counts[(int64_t)blockIdx.x * a.experts + e] = count[e];
}

// Places the routes of this block's part.  Each wave takes a run of them: the
// waves' counts, summed over earlier blocks, experts and waves, are its first
// places, and within 64 routes a route's place is the number of equal keys before it.
__global__ __launch_bounds__(kGroupWaves * kWave) void group_place_kernel(GroupArgs a, int blocks) {
    __shared__ int next[kGroupWaves][kGroupMaxExperts + 1];
    __shared__ int before[kGroupMaxExperts + 1], all[kGroupMaxExperts + 1], sums[kGroupWaves];
    const int lane = lane_id(), wave = threadIdx.x / kWave, n = a.experts;
    const int64_t begin = blockIdx.x * a.part, end = begin + a.part < a.pairs ? begin + a.part : a.pairs;
    const int64_t run = (a.part + kGroupWaves * kWave - 1) / (kGroupWaves * kWave) * kWave;
    const int64_t first = begin + wave * run, last = first + run < end ? first + run : end;
    for (int e = lane; e <= n; e += kWave) next[wave][e] = 0;
    for (int e = threadIdx.x; e <= n; e += blockDim.x) before[e] = all[e] = 0;
    __syncthreads();
    for (int64_t p = first + lane; p < last; p += kWave) atomicAdd(&next[wave][expert_of(a, p, last)], 1);
    // counts of earlier blocks and of all (whole numbers: any order), a thread an expert and
    // every blockDim / n-th block
    if (blocks > 1) {
        const int threads = (int)blockDim.x / n * n, step = threads / n, e = threadIdx.x % n;
        int earlier = 0, sum = 0;
        if ((int)threadIdx.x < threads)
#pragma unroll 8
            for (int b = threadIdx.x / n; b < blocks; b += step) {
                const int c = a.counts[(int64_t)b * n + e];
                sum += c;
                earlier += b < (int)blockIdx.x ? c : 0;
            }
        if (sum) atomicAdd(&all[e], sum);
        if (earlier) atomicAdd(&before[e], earlier);
    }
    __syncthreads();
    // first places: the running sum over experts, 64 a wave
    int mine[(kGroupMaxExperts + kGroupWaves * kWave - 1) / (kGroupWaves * kWave)];
    static_assert(sizeof(mine) == 4, "an expert a thread");
    const int e = threadIdx.x;
    int total = 0;
    if (e < n) {
        if (blocks > 1) total = all[e];
        else
            for (int w = 0; w < kGroupWaves; ++w) total += next[w][e];
    }
    int scan = total;
    for (int d = 1; d < kWave; d *= 2) {
        const int v = __shfl_up(scan, d);
        if (lane >= d) scan += v;
    }
    if (lane == kWave - 1) sums[wave] = scan;
    __syncthreads();
    int start = scan - total;
    for (int w = 0; w < wave; ++w) start += sums[w];
    int present = 0;
    for (int w = 0; w < kGroupWaves; ++w) present += sums[w];
    if (e < n) {
        if (blockIdx.x == 0) a.offsets[e] = start;
        int at = start + (blocks > 1 ? before[e] : 0);
        for (int w = 0; w < kGroupWaves; ++w) {
            const int c = next[w][e];
            next[w][e] = at;
            at += c;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[n] = present;
    // places past the last: each block clears its part of them
    for (int64_t p = begin + threadIdx.x; p < end; p += blockDim.x)
        if (p >= present) a.rows[p] = -1;
    __syncthreads();
    const int bits = 32 - __builtin_clz((unsigned)n);
    for (int64_t from = first; from < last; from += kWave) {
        const int64_t p = from + lane;
        const int key = p < last ? expert_of(a, p, last) : n;
        const uint64_t same = same_key(key, bits);
        const int rank = __popcll(same & ((1ull << lane) - 1));
        const int at = next[wave][key] + rank;
        __builtin_amdgcn_wave_barrier();
        if (rank == 0) next[wave][key] = at + __popcll(same);
        __builtin_amdgcn_wave_barrier();
        if (p < last) {
            a.slots[p] = key < n ? at : -1;
            if (key < n) a.rows[at] = (int)(p / a.routes);
        }
    }
}

}  // namespace

hipError_t launch_group_routes(const loom_launch_config &cfg, const GroupArgs &a, hipStream_t stream) {
    const dim3 grid(cfg.workgroups[0]), block(cfg.workgroup_size[0]);
    if (cfg.workgroups[0] > 1) hipLaunchKernelGGL(group_count_kernel, grid, block, 0, stream, a);
    hipLaunchKernelGGL(group_place_kernel, grid, block, 0, stream, a, (int)cfg.workgroups[0]);
    return hipGetLastError();
}

}  // namespace loom
