// plan_experts.hpp -- (token, expert) pairs sorted by expert, stably: a counting sort.
//
// Pairs are cut into runs, one a workgroup; with several runs a first launch
// counts the experts of each. The placing launch's workgroups each add up the
// counts of all runs, so that there is nothing to wait for between them: the
// experts' offsets, and where their own run's pairs begin. Within a run each
// wave has a stretch of pairs and counters of its own; 64 pairs at a time find
// their rank among equal experts by ballots over the expert number's bits. No
// place depends on the order in which waves or workgroups run.
#pragma once

#include "mx_common.hpp"

namespace qg {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortMaxRuns = 256;

struct SortParams {
    const int32_t *ids;
    int64_t pairs;
    int64_t run;             // pairs of a workgroup, a multiple of 64 * kSortWaves
    int32_t runs, experts, bits;
    int32_t *counts;         // [runs][experts], with several runs
    int32_t *offsets, *order, *slots;
};

// An expert's number, or `experts` for a pair that belongs to none.
__device__ __forceinline__ int sort_key(const SortParams &p, int64_t pair)
{
    const int id = p.ids[pair];
    return id >= 0 && id < p.experts ? id : p.experts;
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortParams p)
{
    extern __shared__ int32_t hist[];                 // [experts + 1]
    for (int e = threadIdx.x; e <= p.experts; e += kSortThreads) hist[e] = 0;
    __syncthreads();
    const int64_t first = blockIdx.x * p.run, last = min(first + p.run, p.pairs);
    for (int64_t i = first + threadIdx.x; i < last; i += kSortThreads) atomicAdd(&hist[sort_key(p, i)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kSortThreads) p.counts[int64_t(blockIdx.x) * p.experts + e] = hist[e];
}

__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortParams p)
{
    // [waves][experts + 1]: first counts, then the next place of each wave's pairs
    extern __shared__ int32_t next[];
    __shared__ int32_t wave_sums[kSortWaves];
    __shared__ int32_t sorted;                        // pairs that belong to an expert
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, width = p.experts + 1;
    for (int i = threadIdx.x; i < kSortWaves * width; i += kSortThreads) next[i] = 0;
    __syncthreads();
    int32_t *mine = next + wave * width;
    const int64_t stretch = p.run / kSortWaves;
    const int64_t first = blockIdx.x * p.run + wave * stretch, last = min(first + stretch, p.pairs);
    for (int64_t i = first + lane; i < last; i += 64) atomicAdd(&mine[sort_key(p, i)], 1);
    __syncthreads();

    // thread e: its expert's pairs in this run, in those before it and in all
    const int e = threadIdx.x;                        // experts <= threads
    int before = 0, all = 0;
    if (e < p.experts) {
        if (p.runs > 1) {
            for (int b = 0; b < p.runs; ++b) {
                const int n = p.counts[int64_t(b) * p.experts + e];
                before += b < static_cast<int>(blockIdx.x) ? n : 0;
                all += n;
            }
        } else {
            for (int w = 0; w < kSortWaves; ++w) all += next[w * width + e];
        }
    }
    const int upto = wave_inclusive_sum32(all);
    if (lane == 63) wave_sums[wave] = upto;
    __syncthreads();
    int start = upto - all;
    for (int w = 0; w < wave; ++w) start += wave_sums[w];
    if (e == kSortThreads - 1) sorted = start + all;
    if (e < p.experts) {
        if (blockIdx.x == 0) {
            p.offsets[e] = start;
            if (e == p.experts - 1) p.offsets[p.experts] = start + all;
        }
        int at = start + before;
        for (int w = 0; w < kSortWaves; ++w) {
            const int n = next[w * width + e];
            next[w * width + e] = at;
            at += n;
        }
    }
    __syncthreads();

    for (int64_t i = first; i < last; i += 64) {      // the same for the whole wave
        const int64_t pair = i + lane;
        const bool real = pair < last;
        const int key = real ? sort_key(p, pair) : p.experts;
        uint64_t same = __ballot(real);               // lanes with this lane's expert
        for (int b = 0; b < p.bits; ++b) {
            const uint64_t set = __ballot((key >> b) & 1);
            same &= (key >> b) & 1 ? set : ~set;
        }
        const int rank = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(same >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(same), 0));
        const bool placed = real && key < p.experts;
        int slot = -1;
        if (placed) slot = mine[key] + rank;
        wave_order();                                 // all have read before the first of each expert counts on
        if (placed && rank == 0) mine[key] = slot + __popcll(same);
        wave_order();
        if (real) p.slots[pair] = slot;
        if (placed) p.order[slot] = static_cast<int32_t>(pair);
    }
    // behind the last sorted pair
    const int64_t rest = p.pairs - sorted;
    for (int64_t i = int64_t(blockIdx.x) * kSortThreads + threadIdx.x; i < rest; i += int64_t(gridDim.x) * kSortThreads)
        p.order[sorted + i] = -1;
}

}  // namespace qg
