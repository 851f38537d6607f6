// attn_join.hpp -- partial results of attention over splits of the tokens
// joined: out = sum_s f_s out_s / sum_s f_s sum_s, f_s = 2^(R_s - R).
#pragma once

#include "attn_common.hpp"

namespace qg {

// Joins the splits of a row and head: WAVES waves of a workgroup of 4 each
// (one where splits are few, four where rows are few and splits many). The
// statistics of the splits are taken a lane each; then runs of D / 4 lanes
// add up the splits s = run, run + runs, ..., and the runs are added in a
// fixed tree. The rows of a tile share their splits, so their count is found
// from the row's tile as the attention kernels do. A chain of latencies (cu_q,
// kv_len, statistics, partial results) of 4 to 6 us, whatever the sizes up to
// some 10 MB of partial results; split counts are chosen with that in mind.
constexpr int kMaxSplits = 256;

template <typename T, int D, int R, int TOK, int WAVES>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnParams p)
{
    constexpr int kLanes = D / 4, kRuns = WAVES * 64 / kLanes;
    __shared__ float weight[4 / WAVES][WAVES == 1 ? 64 : kMaxSplits];
    __shared__ f32x4 sums[WAVES == 1 ? 1 : 4][kLanes];
    __shared__ float red[4][2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int mine = WAVES == 1 ? wave : 0, id = WAVES == 1 ? lane : threadIdx.x;
    const int64_t row = int64_t(blockIdx.x) * (4 / WAVES) + mine;
    if (row >= p.total_q * p.q_heads) return;              // whole waves; never with WAVES = 4
    const int64_t tok = row / p.q_heads;
    const int head = static_cast<int>(row - tok * p.q_heads);
    // the request of this query row: the last that starts at or before it
    int count = 0;
    for (int base = 0; base < p.batch; base += 64) {
        const int b = base + lane;
        const uint64_t m = __ballot(b < p.batch && attn_cu(p, b) <= tok);
        count += __popcll(m);
        if (m != ~0ull) break;
    }
    if (count == 0) return;
    RowTile t;
    t.b = count - 1;
    t.q0 = attn_cu(p, t.b);
    t.n_q = attn_cu(p, t.b + 1) - t.q0;
    if (tok < t.q0 || tok - t.q0 >= t.n_q) return;
    const uint32_t r = static_cast<uint32_t>(tok - t.q0) * p.group + head % p.group;
    tile_tokens(p, t, r / R * R, R);
    const int32_t from = t.lo / TOK * TOK;
    int n = static_cast<int>((int64_t(t.hi) - from + p.chunk - 1) / p.chunk);
    n = t.hi <= from ? 0 : n < p.nsplit ? n : p.nsplit;

    const float *stat = p.part_stat + row * p.nsplit * 2;
    float m = kNoReference, own = 0.0f;
    bool bad = false;                                      // a NaN reference
    if (id < n) {
        m = stat[id * 2];
        own = stat[id * 2 + 1];
        bad = m != m;
    }
    const float ref_own = m;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, lane_xor_f32(m, d));
    bad = __any(bad);
    if constexpr (WAVES > 1) {
        if (lane == 0) red[wave][0] = bad ? __builtin_nanf("") : m;
        __syncthreads();
        m = kNoReference;
        bad = false;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float v = red[w][0];
            bad = bad || v != v;
            m = fmaxf(m, v);
        }
    }
    if (bad) m = __builtin_nanf("");
    const float f = id < n ? __builtin_amdgcn_exp2f(ref_own - m) : 0.0f;
    float sum = f * own;
    if (id < n) weight[mine][id] = f;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += lane_xor_f32(sum, d);
    if constexpr (WAVES > 1) {
        if (lane == 0) red[wave][1] = sum;
        __syncthreads();
        sum = (red[0][1] + red[1][1]) + (red[2][1] + red[3][1]);
    } else {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }

    const int run = id / kLanes, quad = id % kLanes;
    const float *part = p.part_out + row * p.nsplit * D + quad * 4;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int s = run; s < n; s += kRuns) o += weight[mine][s] * *reinterpret_cast<const f32x4 *>(part + int64_t(s) * D);
#pragma unroll
    for (int d = 32; d >= kLanes; d >>= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += lane_xor_f32(o[i], d);
    if constexpr (WAVES > 1) {
        if (lane < kLanes) sums[wave][lane] = o;
        __syncthreads();
        if (threadIdx.x >= kLanes) return;
        o = (sums[0][quad] + sums[1][quad]) + (sums[2][quad] + sums[3][quad]);
    } else if (lane >= kLanes) {
        return;
    }
    store_out4(static_cast<T *>(p.out) + tok * p.out_stride + int64_t(head) * D + quad * 4, o * attn_inverse(t, sum));
    if (p.lse && quad == 0) p.lse[row] = attn_lse(t, m, sum);
}

}  // namespace qg
