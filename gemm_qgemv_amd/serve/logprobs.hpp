// logprobs.hpp -- log probabilities of given tokens, entropy, rank and the
// best alternatives of rows of logits, in one pass over them.
//
// With a running maximum m a lane keeps z = sum e^(x - m) and
// t = sum e^(x - m) (x - m); a new maximum m' scales them by a = e^(m - m'):
// z' = a z, t' = a (t + z (m - m')). Then with z, t, m of the whole row
//   log p[i] = (x[i] - m) - log z,    entropy = log z - t / z.
// m starts at the lowest finite value, so rows and parts of rows of
// -infinity need no test: their terms are 0.
//
// The order of the alternatives (larger logit first, ties by lower index) is
// that of the 64-bit keys argmax_key(x, index). A wave keeps its best 64 keys
// sorted over its lanes; a block of 1024 logits is looked at for them only if
// its maximum passes the last one wanted, which gets rare soon (for the n-th
// block about top / n). The block's candidates, one a lane in rounds, are put
// into the list one by one where they are few, or sorted and merged into it by
// bitonic networks over lanes (DPP and permlane swaps: no LDS round trips).
//
// 1024 rows of 151936 logits (622 MB), the best 5: 118.5 us, 5.25 TB/s, bound by
// HBM; one row, the best 20: 13.2 us, 7.5 without alternatives: two launches and
// the latencies of the networks.
//
// A row is cut into slices over workgroups, each slice into runs of blocks
// over 4 waves; the parts are joined over LDS and, with more than one slice,
// by a second launch, in a fixed order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../csrc/qg_device.hpp"
#include "kv_cache.hpp"

namespace qg {

struct LogprobParams {
    const float *x;
    int64_t ld, rows;
    int32_t vocab;
    const int32_t *ids;
    int top;
    float *logprob, *entropy;
    int32_t *rank, *top_ids;
    float *top_logprobs;
    f32x4 *part;                 // [rows][nslice]: m, z, t, count (as bits)
    uint64_t *part_keys;         // [rows][nslice][top]
    int nslice;
    int32_t slice;               // logits of a slice (a multiple of kLpBlock * kLpWaves)
};

constexpr int kLpThreads = 256;
constexpr int kLpWaves = kLpThreads / 64;
constexpr int kLpQuads = 4;                          // 16-byte loads a lane has in flight
constexpr int kLpBlock = 64 * 4 * kLpQuads;          // logits a wave takes at a time
// Candidates of a round that are put into the list one by one; more are sorted
// and merged (27 exchange steps). 1024 rows of 151936, the best 32: 147 us with 8,
// 150 with 4, 148 with 16, 181 with none.
constexpr int kLpFew = 8;
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.44269504088896340736f;

struct Moments {
    float m, z, t;
};

__device__ __forceinline__ Moments lp_join(Moments a, Moments b)
{
    const float m = fmaxf(a.m, b.m);
    const float fa = __builtin_amdgcn_exp2f((a.m - m) * kLog2e), fb = __builtin_amdgcn_exp2f((b.m - m) * kLog2e);
    // an infinite difference of maxima belongs to a side that scales to 0
    const float da = fmaxf(a.m - m, -1000.0f), db = fmaxf(b.m - m, -1000.0f);
    return {m, fmaf(fa, a.z, fb * b.z), fmaf(fa, fmaf(a.z, da, a.t), fb * fmaf(b.z, db, b.t))};
}

// Value of lane ^ D by DPP (D = 1, 2, 4, 8: no LDS round trip).
template <int D>
__device__ __forceinline__ uint32_t near_u32(uint32_t v)
{
    static_assert(D == 1 || D == 2 || D == 4 || D == 8, "within 16 lanes");
    if constexpr (D == 4) {
        // mirrored within 8 lanes (lane ^ 7), then within 4 (lane ^ 3)
        v = __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, false);
        return __builtin_amdgcn_update_dpp(0, v, 0x1B, 0xF, 0xF, false);
    } else {
        constexpr int ctrl = D == 1 ? 0xB1 : D == 2 ? 0x4E : 0x128;
        return __builtin_amdgcn_update_dpp(0, v, ctrl, 0xF, 0xF, false);
    }
}

// The larger (or the smaller) of a lane's key and that of lane ^ D.
template <int D>
__device__ __forceinline__ uint64_t exchange(uint64_t k, bool keep_max)
{
    const uint32_t lo = static_cast<uint32_t>(k), hi = static_cast<uint32_t>(k >> 32);
    uint64_t a, b;
    if constexpr (D <= 8) {
        a = k;
        b = (static_cast<uint64_t>(near_u32<D>(hi)) << 32) | near_u32<D>(lo);
    } else {
        // both partners get the same pair: the swaps return it in either lane
        const auto rl = D == 16 ? __builtin_amdgcn_permlane16_swap(lo, lo, false, false) : __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
        const auto rh = D == 16 ? __builtin_amdgcn_permlane16_swap(hi, hi, false, false) : __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
        a = (static_cast<uint64_t>(rh[0]) << 32) | rl[0];
        b = (static_cast<uint64_t>(rh[1]) << 32) | rl[1];
    }
    return (a > b) == keep_max ? a : b;
}

// One run of exchange steps W / 2, .., 1 of a bitonic network over the 64
// lanes; lanes of runs of W in turn sort down and up (W = 64: all down).
template <int W, int D>
__device__ __forceinline__ uint64_t bitonic_steps(uint64_t k, int lane)
{
    if constexpr (D >= 1) {
        k = exchange<D>(k, ((lane & D) == 0) == ((lane & W) == 0));
        return bitonic_steps<W, D / 2>(k, lane);
    } else {
        return k;
    }
}

// Any 64 keys into descending order over the lanes.
__device__ __forceinline__ uint64_t bitonic_sort(uint64_t k, int lane)
{
    k = bitonic_steps<2, 1>(k, lane);
    k = bitonic_steps<4, 2>(k, lane);
    k = bitonic_steps<8, 4>(k, lane);
    k = bitonic_steps<16, 8>(k, lane);
    k = bitonic_steps<32, 16>(k, lane);
    return bitonic_steps<64, 32>(k, lane);
}

// The 64 largest of a descending and an ascending list, descending.
__device__ __forceinline__ uint64_t merge_lists(uint64_t down, uint64_t up, int lane)
{
    return bitonic_steps<64, 32>(down > up ? down : up, lane);
}

__device__ __forceinline__ uint64_t lane_u64(uint64_t v, int src)
{
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(v), src);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(v >> 32), src);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// A key put into its place in a descending list (the last one falls out).
__device__ __forceinline__ uint64_t insert_key(uint64_t list, uint64_t key, int lane)
{
    const int place = __popcll(__ballot(list > key));
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<uint32_t>(list), 0x138, 0xF, 0xF, false);          // lane - 1's
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<uint32_t>(list >> 32), 0x138, 0xF, 0xF, false);
    const uint64_t before = (static_cast<uint64_t>(hi) << 32) | lo;
    return lane < place ? list : lane == place ? key : before;
}

__device__ __forceinline__ float key_value(uint64_t key)
{
    const uint32_t u = static_cast<uint32_t>(key >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

// Joined with lane ^ d's; both partners add in the same order.
__device__ __forceinline__ void lp_join_lanes(Moments &mo, int lane, int d)
{
    const Moments o = {lane_xor_f32(mo.m, d), lane_xor_f32(mo.z, d), lane_xor_f32(mo.t, d)};
    mo = lane & d ? lp_join(o, mo) : lp_join(mo, o);
}

struct RowResult {
    Moments mo;
    int32_t before;              // tokens before the given one
    uint64_t list;               // lane i: the i-th best key
};

// The results of the workgroup's WAVES waves joined (the list: in wave 0).
template <int WAVES>
__device__ __forceinline__ RowResult lp_join_waves(RowResult r, bool want_top)
{
    __shared__ f32x4 stat[WAVES];
    __shared__ uint64_t lists[WAVES][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane == 0) stat[wave] = f32x4{r.mo.m, r.mo.z, r.mo.t, __int_as_float(r.before)};
    if (want_top) {
        // halves of the waves hand their lists to the other halves
#pragma unroll
        for (int n = WAVES / 2; n >= 1; n >>= 1) {
            if (wave >= n && wave < 2 * n) lists[wave][lane] = r.list;
            __syncthreads();
            if (wave < n) r.list = merge_lists(r.list, lists[wave + n][63 - lane], lane);
        }
    } else {
        __syncthreads();
    }
    // a wave's statistics in a lane, joined by halves (every lane gets them)
    const f32x4 mine = stat[lane & (WAVES - 1)];
    RowResult o;
    o.mo = {mine[0], mine[1], mine[2]};
    o.before = __float_as_int(mine[3]);
    o.list = r.list;
#pragma unroll
    for (int d = WAVES / 2; d >= 1; d >>= 1) {
        lp_join_lanes(o.mo, lane, d);
        o.before += __float_as_int(lane_xor_f32(__int_as_float(o.before), d));
    }
    return o;
}

// Results of a whole row written (by wave 0).
__device__ __forceinline__ void lp_finish(const LogprobParams &p, int64_t row, const RowResult &r)
{
    const int lane = threadIdx.x & 63;
    if (threadIdx.x >= 64) return;
    const float nan = __builtin_nanf("");
    const float log_z = r.mo.z > 0.0f ? logf(r.mo.z) : nan;      // NaN too where z is NaN
    if (lane == 0) {
        if (p.entropy) p.entropy[row] = log_z - r.mo.t / r.mo.z;
        if (p.ids) {
            const int32_t id = p.ids[row];
            const bool in = id >= 0 && id < p.vocab;
            if (p.logprob) p.logprob[row] = in ? (p.x[row * p.ld + id] - r.mo.m) - log_z : nan;
            if (p.rank) p.rank[row] = in ? r.before + 1 : 0;
        }
    }
    if (lane < p.top) {
        // fewer keys than `top` only where the row holds NaNs
        const uint32_t id = argmax_key_index(r.list);
        p.top_ids[row * p.top + lane] = static_cast<int32_t>(id < static_cast<uint32_t>(p.vocab) ? id : 0);
        p.top_logprobs[row * p.top + lane] = (key_value(r.list) - r.mo.m) - log_z;
    }
}

__global__ __launch_bounds__(kLpThreads) void logprob_kernel(LogprobParams p)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = blockIdx.x / static_cast<unsigned>(p.nslice);
    const int slice = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.nslice));
    const float *x = p.x + row * p.ld;
    // positions count from the 16-byte boundary at or before the row's start
    const int32_t skew = static_cast<int32_t>((reinterpret_cast<uintptr_t>(x) >> 2) & 3);
    const int64_t span = int64_t(p.vocab) + skew;
    const int64_t begin = int64_t(slice) * p.slice + int64_t(wave) * (p.slice / kLpWaves);
    int64_t end = begin + p.slice / kLpWaves;
    end = end < span ? end : span;

    int32_t id = -1;
    float given = 0.0f;
    if (p.ids) {
        id = p.ids[row];
        if (id < 0 || id >= p.vocab) id = -1;
        else given = x[id];
    }
    const int top = p.top;
    RowResult r;
    r.mo = {kLowest, 0.0f, 0.0f};
    r.before = 0;
    r.list = 0;
    uint64_t last_key = 0;                 // the worst key wanted so far (0: the list is not full)
    float last = 0.0f;

    for (int64_t base = begin; base < end; base += kLpBlock) {
        // the index of element e of quad j: at(j) + e
        auto at = [&](int j) { return static_cast<int32_t>(base + j * 256 - skew) + lane * 4; };
        const bool inner = base >= skew && base + kLpBlock <= span;
        f32x4 v[kLpQuads];
        if (inner) {
#pragma unroll
            for (int j = 0; j < kLpQuads; ++j) v[j] = *reinterpret_cast<const f32x4 *>(x + at(j));
        } else {
#pragma unroll
            for (int j = 0; j < kLpQuads; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int32_t i = at(j) + e;
                    v[j][e] = i >= 0 && i < p.vocab ? x[i] : -__builtin_inff();
                }
        }
        float bm = v[0][0];
#pragma unroll
        for (int j = 0; j < kLpQuads; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) bm = fmaxf(bm, v[j][e]);

        const float m = fmaxf(r.mo.m, bm);
        const float a = __builtin_amdgcn_exp2f((r.mo.m - m) * kLog2e), da = fmaxf(r.mo.m - m, -1000.0f);
        r.mo.t = a * fmaf(r.mo.z, da, r.mo.t);
        r.mo.z *= a;
        r.mo.m = m;
#pragma unroll
        for (int j = 0; j < kLpQuads; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float d = v[j][e] - m;
                const float w = __builtin_amdgcn_exp2f(d * kLog2e);
                r.mo.z += w;
                r.mo.t = fmaf(w, fmaxf(d, -1000.0f), r.mo.t);     // -infinity: 0 * -1000
            }

        if (id >= 0) {
            const int32_t lo = static_cast<int32_t>(base - skew);
            if (inner && lo + kLpBlock <= id) {
#pragma unroll
                for (int j = 0; j < kLpQuads; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) r.before += __popcll(__ballot(v[j][e] >= given));
            } else if (inner && lo > id) {
#pragma unroll
                for (int j = 0; j < kLpQuads; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) r.before += __popcll(__ballot(v[j][e] > given));
            } else {
#pragma unroll
                for (int j = 0; j < kLpQuads; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int32_t i = at(j) + e;
                        const bool in = i >= 0 && i < p.vocab;
                        r.before += __popcll(__ballot(in && (v[j][e] > given || (v[j][e] == given && i < id))));
                    }
            }
        }

        if (top > 0 && (last_key == 0 || __any(bm > last))) {
            // the block's values in their order (0: not of the row, or taken)
            uint32_t order[4 * kLpQuads];
#pragma unroll
            for (int j = 0; j < kLpQuads; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int32_t i = at(j) + e;
                    order[j * 4 + e] = inner || (i >= 0 && i < p.vocab) ? float_order_bits(v[j][e]) : 0;
                }
            // a lane's best value that is left, in rounds until none passes the list's last
            for (;;) {
                uint32_t best = order[0];
                int slot = 0;
#pragma unroll
                for (int n = 1; n < 4 * kLpQuads; ++n) {
                    slot = order[n] > best ? n : slot;           // the first of equal ones
                    best = order[n] > best ? order[n] : best;
                }
                const uint32_t index = static_cast<uint32_t>(at(slot >> 2) + (slot & 3));
                const uint64_t key = best ? (static_cast<uint64_t>(best) << 32) | (0xFFFFFFFFu - index) : 0;
                const bool passes = key > last_key;
                uint64_t in = __ballot(passes);
                if (in == 0) break;
#pragma unroll
                for (int n = 0; n < 4 * kLpQuads; ++n) order[n] = n == slot ? 0 : order[n];
                if (__popcll(in) > kLpFew) {
                    r.list = merge_lists(r.list, shfl_xor_u64(bitonic_sort(passes ? key : 0, lane), 63), lane);
                    last_key = lane_u64(r.list, top - 1);
                } else {
                    for (; in != 0; in &= in - 1) {
                        const uint64_t k = lane_u64(key, __builtin_ctzll(in));
                        if (k <= last_key) continue;             // an earlier one has raised the bar
                        r.list = insert_key(r.list, k, lane);
                        last_key = lane_u64(r.list, top - 1);
                    }
                }
                last = key_value(last_key);
            }
        }
    }

    // lanes joined
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) lp_join_lanes(r.mo, lane, d);
    r = lp_join_waves<kLpWaves>(r, top > 0);
    if (p.nslice == 1) {
        lp_finish(p, row, r);
    } else if (wave == 0) {
        if (lane == 0) p.part[blockIdx.x] = f32x4{r.mo.m, r.mo.z, r.mo.t, __int_as_float(r.before)};
        if (lane < top) p.part_keys[int64_t(blockIdx.x) * top + lane] = r.list;
    }
}

// Joins the slices of a row.
constexpr int kLpJoinThreads = 1024;

__global__ __launch_bounds__(kLpJoinThreads) void logprob_join_kernel(LogprobParams p)
{
    constexpr int kWaves = kLpJoinThreads / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x;
    RowResult r;
    r.mo = {kLowest, 0.0f, 0.0f};
    r.before = 0;
    r.list = 0;
    // a few slices' results are asked for before the first is used
    constexpr int kAhead = 4;
    for (int s0 = wave; s0 < p.nslice; s0 += kWaves * kAhead) {
        f32x4 v[kAhead];
        uint64_t list[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int s = s0 + j * kWaves;
            const int64_t at = row * p.nslice + (s < p.nslice ? s : s0);
            v[j] = p.part[at];
            list[j] = 63 - lane < p.top ? p.part_keys[at * p.top + 63 - lane] : 0;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (s0 + j * kWaves >= p.nslice) break;
            r.mo = lp_join(r.mo, {v[j][0], v[j][1], v[j][2]});
            r.before += __float_as_int(v[j][3]);
            if (p.top > 0) r.list = merge_lists(r.list, list[j], lane);
        }
    }
    r = lp_join_waves<kWaves>(r, p.top > 0);
    lp_finish(p, row, r);
}

}  // namespace qg
