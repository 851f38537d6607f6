// plan_experts.hpp -- (token, expert) pairs sorted by expert, stably: a counting sort.
//
// Pairs are cut into runs, one a workgroup; with several runs a first launch
// counts the experts of each. The placing launch's workgroups each add up the
// counts of all runs, so that there is nothing to wait for between them: the
// experts' offsets, and where their own run's pairs begin. Within a run each
// wave has a stretch of pairs and counters of its own; 64 pairs at a time find
// their rank among equal experts by ballots over the expert number's bits. No
// place depends on the order in which waves or workgroups run. Bound by
// latencies: 98466 pairs, 256 experts, 4 us to count and 7.5 to place (13 in runs of
// twice the length, each expert's counts added up by one thread).
#pragma once

#include "mx_common.hpp"

namespace qg {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortMaxRuns = 256;
constexpr int kSortSteps = 2;        // of 64 pairs that a wave keeps in registers, and takes unless runs are many

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

// LDS of a placing workgroup: [waves][experts + 1] first counts, then the next place of
// each wave's pairs; then the sums over runs, and the waves'.
constexpr int sort_place_ints(int experts) { return kSortWaves * (experts + 1) + 2 * kSortThreads + kSortWaves + 1; }

__device__ __forceinline__ void sort_place(const SortParams &p, int32_t *next)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, width = p.experts + 1;
    int32_t *sums = next + kSortWaves * width, *wave_sums = sums + 2 * kSortThreads, *sorted = wave_sums + kSortWaves;
    for (int i = threadIdx.x; i < kSortWaves * width; i += kSortThreads) next[i] = 0;
    // With several runs: thread (q, e) adds up the counts of expert e of every Qth run
    // from q on, those of runs before this one and all.
    int bits = 6;
    while ((1 << bits) < p.experts) ++bits;
    const int parts = kSortThreads >> bits, e = threadIdx.x & ((1 << bits) - 1), part = threadIdx.x >> bits;
    int before = 0, all = 0;
    if (p.runs > 1 && e < p.experts) {
#pragma unroll 8
        for (int b = part; b < p.runs; b += parts) {
            const int n = p.counts[b * p.experts + e];
            before += b < static_cast<int>(blockIdx.x) ? n : 0;
            all += n;
        }
    }
    int32_t *mine = next + wave * width;
    const int64_t stretch = p.run / kSortWaves;
    const int64_t first = blockIdx.x * p.run + wave * stretch, last = min(first + stretch, p.pairs);
    int keys[kSortSteps];
#pragma unroll
    for (int s = 0; s < kSortSteps; ++s) keys[s] = first + 64 * s + lane < last ? sort_key(p, first + 64 * s + lane) : -1;
    sums[threadIdx.x] = before;
    sums[kSortThreads + threadIdx.x] = all;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kSortSteps; ++s)
        if (keys[s] >= 0) atomicAdd(&mine[keys[s]], 1);
    for (int64_t i = first + 64 * kSortSteps + lane; i < last; i += 64) atomicAdd(&mine[sort_key(p, i)], 1);
    __syncthreads();

    // thread e: its expert's pairs in this run, in those before it and in all
    before = all = 0;
    if (threadIdx.x < p.experts) {
        if (p.runs > 1)
            for (int q = 0; q < parts; ++q) {
                before += sums[(q << bits) + threadIdx.x];
                all += sums[kSortThreads + (q << bits) + threadIdx.x];
            }
        else
            for (int w = 0; w < kSortWaves; ++w) all += next[w * width + threadIdx.x];
    }
    const int upto = wave_inclusive_sum32(all);
    if (lane == 63) wave_sums[wave] = upto;
    __syncthreads();
    int start = upto - all;
    for (int w = 0; w < wave; ++w) start += wave_sums[w];
    if (threadIdx.x == kSortThreads - 1) *sorted = start + all;      // (experts <= threads)
    if (threadIdx.x < p.experts) {
        if (blockIdx.x == 0) {
            p.offsets[threadIdx.x] = start;
            if (threadIdx.x == p.experts - 1) p.offsets[p.experts] = start + all;
        }
        int at = start + before;
        for (int w = 0; w < kSortWaves; ++w) {
            const int n = next[w * width + threadIdx.x];
            next[w * width + threadIdx.x] = at;
            at += n;
        }
    }
    __syncthreads();

    const auto step = [&](int64_t pair, int key) __attribute__((always_inline)) {        // key -1: behind the stretch
        const bool real = key >= 0;
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
    };
#pragma unroll
    for (int s = 0; s < kSortSteps; ++s) step(first + 64 * s + lane, keys[s]);
    for (int64_t i = first + 64 * kSortSteps; i < last; i += 64)      // the same for the whole wave
        step(i + lane, i + lane < last ? sort_key(p, i + lane) : -1);
    // behind the last sorted pair
    const int64_t rest = p.pairs - *sorted;
    for (int64_t i = int64_t(blockIdx.x) * kSortThreads + threadIdx.x; i < rest; i += int64_t(gridDim.x) * kSortThreads)
        p.order[*sorted + i] = -1;
}

__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortParams p)
{
    extern __shared__ int32_t lds[];
    sort_place(p, lds);
}

}  // namespace qg
