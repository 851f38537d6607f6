// plan.hpp -- pages, lengths, row starts and slots of a step, from lengths.
//
// A few thousand integer operations: the floor is one launch (4.1 us for 64
// decoding requests and 6.4 for 512 with 65536 new tokens, replayed from a
// graph: a launch and a chain of loads, lengths, ring counts, ring entry).
// Every workgroup computes the running sums over all requests itself (a few
// hundred cycles; the requests' lengths come from L2) and then fills its share
// of the slots, of the pages taken or of those given back (three rows of
// workgroups, so that the three latencies do not add up). So there is one
// launch, no workspace, and nothing for one workgroup to wait for in another.
// That needs two rules of the operator: pages given back in a call are not
// taken in the same call (takers read ring entries head..tail-1, givers write
// from tail on), and the new ring counts go to another place than the old ones.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qg {

struct PlanParams {
    const int32_t *len_old, *keep, *n_new;
    int batch, page_shift;
    int32_t *table;
    int64_t table_stride;
    int32_t *ring;
    int64_t ring_size;
    const int64_t *state_in;
    int64_t *state_out;
    int32_t *kv_len, *cu_q, *slots, *pos;
    int64_t total;
    int32_t *denied;
};

constexpr int kPlanThreads = 256;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int64_t kPlanMaxLen = int64_t(1) << 30;

// What one request holds, keeps and wants (pages: those within its table row).
struct PlanRequest {
    int32_t keep, n_new;
    int64_t have, kept, want;
    bool fits;       // its pages fit its row of the table
    int64_t grow;
};

__device__ __forceinline__ PlanRequest plan_request(const PlanParams &p, int b)
{
    auto clamp = [](int64_t v, int64_t hi) { return v < 0 ? 0 : v > hi ? hi : v; };
    const int64_t old = clamp(p.len_old[b], kPlanMaxLen);
    PlanRequest r;
    r.keep = static_cast<int32_t>(clamp(p.keep[b], old));
    r.n_new = static_cast<int32_t>(clamp(p.n_new[b], kPlanMaxLen));
    const int64_t round = (int64_t(1) << p.page_shift) - 1;
    r.have = clamp((old + round) >> p.page_shift, p.table_stride);
    r.kept = clamp((r.keep + round) >> p.page_shift, p.table_stride);
    r.want = (int64_t(r.keep) + r.n_new + round) >> p.page_shift;
    r.fits = r.want <= p.table_stride;
    r.grow = r.fits && r.want > r.have ? r.want - r.have : 0;
    return r;
}

// v plus the value DPP brings from a lower lane (0 where there is none).
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t add_from(int64_t v)
{
    const int lo = static_cast<int>(v), hi = static_cast<int>(v >> 32);
    const uint32_t l = __builtin_amdgcn_update_dpp(0, lo, CTRL, ROWS, 0xF, false);
    const int32_t h = __builtin_amdgcn_update_dpp(0, hi, CTRL, ROWS, 0xF, false);
    return v + ((static_cast<int64_t>(h) << 32) | l);
}

// Inclusive sum over the lanes of a wave (shifts within 16 lanes, then the
// last lane of a row, and of half a wave, broadcast to what follows).
__device__ __forceinline__ int64_t wave_inclusive_sum(int64_t v)
{
    v = add_from<0x111, 0xF>(v);
    v = add_from<0x112, 0xF>(v);
    v = add_from<0x114, 0xF>(v);
    v = add_from<0x118, 0xF>(v);
    v = add_from<0x142, 0xA>(v);
    return add_from<0x143, 0xC>(v);
}

// Exclusive sums over the workgroup's threads of two values a thread; the
// totals are those of all. `parts` is LDS used once.
__device__ __forceinline__ void block_exclusive_sums(int64_t (&v)[2], int64_t (&total)[2], int64_t (&parts)[2][kPlanWaves])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t run[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        run[k] = wave_inclusive_sum(v[k]);
        if (lane == 63) parts[k][wave] = run[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        int64_t before = 0;
        total[k] = 0;
#pragma unroll
        for (int w = 0; w < kPlanWaves; ++w) {
            if (w < wave) before += parts[k][w];
            total[k] += parts[k][w];
        }
        v[k] = before + run[k] - v[k];
    }
}

// count mod size, 0 <= result < size < 2^31 (a 64-bit division takes longer
// than the rest of a small plan).
__device__ __forceinline__ int64_t ring_place(int64_t count, int64_t size)
{
    constexpr int64_t kExact = int64_t(1) << 52;
    int64_t m;
    if (count < kExact && count > -kExact) {
        m = count - static_cast<int64_t>(static_cast<double>(count) / static_cast<double>(size)) * size;   // off by one size at most
    } else {
        m = count % size;
    }
    if (m < 0) m += size;
    return m < size ? m : m - size;
}

__device__ __forceinline__ int32_t saturate(int64_t v) { return v > 0x7fffffff ? 0x7fffffff : static_cast<int32_t>(v); }

// Last b of starts[0..n) with starts[b] <= v (starts[0] <= v, not decreasing).
__device__ __forceinline__ int last_not_above(const int32_t *starts, int n, int64_t v)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kPlanThreads) void kv_plan_kernel(PlanParams p)
{
    extern __shared__ int32_t lds[];
    int32_t *cu = lds, *take_at = cu + p.batch + 1, *give_at = take_at + p.batch;
    __shared__ int64_t parts[2][2][kPlanWaves];
    const int B = p.batch, per = (B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(int(threadIdx.x) * per, B), b1 = min(b0 + per, B);
    const bool first_block = blockIdx.x == 0 && blockIdx.y == 0;
    const int64_t head = p.state_in[0], tail = p.state_in[1];
    const int64_t avail = tail - head > p.ring_size ? p.ring_size : tail - head;

    int64_t sums[2] = {0, 0}, totals[2];
    for (int b = b0; b < b1; ++b) {
        const PlanRequest r = plan_request(p, b);
        sums[0] += r.n_new;
        sums[1] += r.grow;
    }
    block_exclusive_sums(sums, totals, parts[0]);
    int64_t rows = sums[0], grow = sums[1];
    const int64_t all_rows = totals[0];
    // granted requests that grow come before the denied ones that grow, so
    // the running sum of `grow` is also that of the pages taken
    int64_t give = 0, taken = 0;
    int denied = 0;
    for (int b = b0; b < b1; ++b) {
        const PlanRequest r = plan_request(p, b);
        const bool granted = r.fits && (r.grow == 0 || grow + r.grow <= avail);
        cu[b] = saturate(rows);
        take_at[b] = saturate(grow);
        const int64_t after = granted ? r.want : r.kept;
        give += r.have > after ? r.have - after : 0;
        if (granted) taken += r.grow;
        else ++denied;
        if (first_block) {
            p.cu_q[b] = saturate(rows);
            p.kv_len[b] = saturate(int64_t(r.keep) + (granted ? r.n_new : 0));
        }
        rows += r.n_new;
        grow += r.grow;
    }
    sums[0] = give;
    sums[1] = (taken << 16) + denied;      // two small counts in one sum
    block_exclusive_sums(sums, totals, parts[1]);
    int64_t at = sums[0];
    const int64_t all_give = totals[0], all_taken = totals[1] >> 16;
    for (int b = b0; b < b1; ++b) {
        const PlanRequest r = plan_request(p, b);
        const bool granted = r.fits && (r.grow == 0 || take_at[b] + r.grow <= avail);
        give_at[b] = saturate(at);
        const int64_t after = granted ? r.want : r.kept;
        at += r.have > after ? r.have - after : 0;
    }
    if (threadIdx.x == 0) {
        cu[B] = saturate(all_rows);
        if (first_block) {
            p.cu_q[B] = saturate(all_rows);
            p.state_out[0] = head + all_taken;
            p.state_out[1] = tail + all_give;
            p.denied[0] = static_cast<int32_t>(totals[1] & 0xffff);
        }
    }
    __syncthreads();

    // places in the ring of its entries head + i and tail + i
    const int64_t front = ring_place(head, p.ring_size), back = ring_place(tail, p.ring_size);
    auto ring_at = [&](int64_t from, int64_t i) {
        const int64_t m = from + (i < p.ring_size ? i : i % p.ring_size);
        return m < p.ring_size ? m : m - p.ring_size;
    };
    const int64_t first = int64_t(blockIdx.x) * kPlanThreads + threadIdx.x, step = int64_t(gridDim.x) * kPlanThreads;
    // pages taken (blockIdx.y 1): entry i of the ring's front is page
    // i - take_at of its request
    for (int64_t i = first; blockIdx.y == 1 && i < all_taken; i += step) {
        const int b = last_not_above(take_at, B, i);
        const PlanRequest r = plan_request(p, b);
        const int64_t col = r.have + (i - take_at[b]);
        if (col < r.want && col < p.table_stride) p.table[b * p.table_stride + col] = p.ring[ring_at(front, i)];
    }
    // pages given back (blockIdx.y 2)
    for (int64_t i = first; blockIdx.y == 2 && i < all_give; i += step) {
        const int b = last_not_above(give_at, B, i);
        const PlanRequest r = plan_request(p, b);
        const bool granted = r.fits && (r.grow == 0 || take_at[b] + r.grow <= avail);
        const int64_t col = (granted ? r.want : r.kept) + (i - give_at[b]);
        if (col < r.have) p.ring[ring_at(back, i)] = p.table[b * p.table_stride + col];
    }
    // slots and positions of the new tokens (blockIdx.y 0; pages taken in this
    // call are read from the ring: their table entries may not be written yet)
    for (int64_t t = first; blockIdx.y == 0 && t < p.total; t += step) {
        int32_t slot = -1, pos = -1;
        if (t < cu[B]) {
            const int b = last_not_above(cu, B, t);
            const PlanRequest r = plan_request(p, b);
            const int64_t at_pos = r.keep + (t - cu[b]);
            pos = saturate(at_pos);
            if (r.fits && (r.grow == 0 || take_at[b] + r.grow <= avail)) {
                const int64_t col = at_pos >> p.page_shift;
                const int64_t page = col < r.have ? p.table[b * p.table_stride + col]
                                                  : p.ring[ring_at(front, take_at[b] + (col - r.have))];
                const int64_t place = page * (int64_t(1) << p.page_shift) + (at_pos & ((int64_t(1) << p.page_shift) - 1));
                if (place == static_cast<int32_t>(place)) slot = static_cast<int32_t>(place);    // or it would be another page's
            }
        }
        p.slots[t] = slot;
        p.pos[t] = pos;
    }
}

}  // namespace qg
