// route.hpp -- a router's rows of logits: the best experts of each and their
// softmax weights.
//
// 16 lanes take a row (one DPP row: maxima over it need no LDS), a lane every
// 16th logit as an order-preserving integer, 0 for what cannot be chosen. Each
// of the `top` rounds takes the largest number by four DPP maxima, then the
// lowest index that has it by four minima. Bound by these rounds, not by memory: 8
// steps that wait for one another behind two passes over a lane's logits (vector
// instructions issue 43% of the time); 16411 x 256 bf16, 6 each, 13.6 us for 9 MB. (Lanes that sort their logits in a
// network first took three times as long: the conditions held for 16 numbers
// at once do not fit in the scalar registers.)
#pragma once

#include "plan_experts.hpp"

namespace qg {

constexpr int kRouteThreads = 256;
constexpr int kRouteRows = kRouteThreads / 16;      // rows of a workgroup

struct RouteParams {
    const void *x;
    int64_t ld;
    int64_t rows;
    int32_t experts, top;
    bool renorm;
    int32_t *ids;
    float *weights;
};

// Over the 16 lanes of a DPP row, in every lane.
template <typename F>
__device__ __forceinline__ uint32_t row16(uint32_t v, F f)
{
    v = f(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0xB1, 0xF, 0xF, false)));
    v = f(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x4E, 0xF, 0xF, false)));
    v = f(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x124, 0xF, 0xF, false)));
    return f(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x128, 0xF, 0xF, false)));
}
__device__ __forceinline__ uint32_t row16_max(uint32_t v) { return row16(v, [](uint32_t a, uint32_t b) { return max(a, b); }); }
__device__ __forceinline__ uint32_t row16_min(uint32_t v) { return row16(v, [](uint32_t a, uint32_t b) { return min(a, b); }); }
__device__ __forceinline__ float row16_sum(float v)
{
    return __uint_as_float(row16(__float_as_uint(v), [](uint32_t a, uint32_t b) { return __float_as_uint(__uint_as_float(a) + __uint_as_float(b)); }));
}

// The float32 that float_order_bits made `u` of.
__device__ __forceinline__ float from_order_bits(uint32_t u)
{
    return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}

// 16 lanes' row. V: logits a lane (16 V >= experts).
template <typename T, int V>
__device__ __forceinline__ void route_row(const RouteParams &p, int64_t row)
{
    const int sub = threadIdx.x & 15;
    const T *x = static_cast<const T *>(p.x) + row * p.ld;
    T t[V];
    // (under no condition, so that all are on their way together)
#pragma unroll
    for (int v = 0; v < V; ++v) t[v] = x[min(v * 16 + sub, p.experts - 1)];
    uint32_t key[V];
    bool bad = false;                                 // a NaN or +infinity
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 16 + sub;
        uint32_t bits;
        if constexpr (sizeof(T) == 4)
            bits = __float_as_uint(t[v]);
        else
            bits = static_cast<uint32_t>(t[v]) << 16;
        if (e >= p.experts) bits = 0xff800000u;       // -infinity
        const bool none = bits == 0xff800000u;
        bad |= !none && (bits & 0x7fffffffu) >= 0x7f800000u;
        key[v] = none ? 0 : float_order_bits(__uint_as_float(bits));
    }
    bad = row16_max(bad) != 0;

    uint32_t best = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) best = max(best, key[v]);
    best = row16_max(best);
    const float m = best ? from_order_bits(best) : 0.0f;
    float z = 0.0f;
    if (!p.renorm) {
#pragma unroll
        for (int v = 0; v < V; ++v) z += key[v] ? expf(from_order_bits(key[v]) - m) : 0.0f;
        z = row16_sum(z);
    }

    constexpr int H = 2;                              // a lane keeps choices sub and sub + 16
    uint32_t got[H] = {0, 0};
    int id[H] = {-1, -1};
    for (int j = 0; j < p.top; ++j) {
        uint32_t mine = 0;
        int at = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (key[v] > mine) mine = key[v], at = v;  // the first of equal ones
        const uint32_t most = row16_max(mine);
        if (most == 0) break;                         // a lane's 15 neighbours leave with it
        const uint32_t e = row16_min(mine == most ? static_cast<uint32_t>(at * 16 + sub) : ~0u);
        const bool won = (e & 15) == static_cast<uint32_t>(sub);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (won && static_cast<uint32_t>(v) == e >> 4) key[v] = 0;
        if (sub == (j & 15)) {
            if (j < 16) got[0] = most, id[0] = static_cast<int>(e);
            else got[1] = most, id[1] = static_cast<int>(e);
        }
    }
    float w[H];
#pragma unroll
    for (int h = 0; h < H; ++h) w[h] = id[h] >= 0 ? expf(from_order_bits(got[h]) - m) : 0.0f;
    if (p.renorm) z = row16_sum(w[0] + w[1]);
    // (one quotient a row: a weight has a rounding more than by a quotient of its own, beside
    // those of its exponential and of the sum)
    const float inv = 1.0f / (z > 0.0f ? z : 1.0f);
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const int j = h * 16 + sub;
        if (j < p.top) {
            p.ids[row * p.top + j] = bad ? -1 : id[h];
            p.weights[row * p.top + j] = bad ? __builtin_nanf("") : w[h] * inv;
        }
    }
}

template <typename T, int V>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteParams p)
{
    const int64_t row = int64_t(blockIdx.x) * kRouteRows + (threadIdx.x >> 4);
    if (row < p.rows) route_row<T, V>(p, row);        // (16 lanes alike)
}

// Router and sort of what one workgroup takes, in one launch (64 x 128, 8 each: 9.2 us
// of latencies against 4.8 and 5.4 in two).
constexpr int kRouteSortRows = kSortThreads / 16;

template <typename T, int V>
__global__ __launch_bounds__(kSortThreads) void route_sort_kernel(RouteParams p, SortParams s)
{
    extern __shared__ int32_t lds[];
    const int row = threadIdx.x >> 4;
    if (row < p.rows) route_row<T, V>(p, row);
    __syncthreads();                                  // the ids are there for all of the workgroup
    sort_place(s, lds);
}

}  // namespace qg
