// combine.hpp -- the experts' rows back to their tokens, with the router's
// weights: out[n] = sum over j of weights[n][j] * y[slots[n][j]], in float32
// and in the order of j. Bound by HBM: every chosen row is read once, four of a token's
// under way together (16411 x 8 rows of 2048 bf16: 105 us, 4.7 TB/s).
#pragma once

#include "mx_common.hpp"

namespace qg {

constexpr int kCombineThreads = 256;

struct CombineParams {
    const void *y;
    const int32_t *slots;
    const float *weights;
    void *out;
    int64_t M, pairs;
    int32_t top;
    uint32_t pieces;         // (token, run of 8 outputs) pairs of this launch
    FastDiv per_row;         // runs of a token
};

// Eight elements side by side, or what there is of them.
template <bool VEC, typename T>
__device__ __forceinline__ void fetch8(const T *src, int n, float (&x)[8])
{
    if constexpr (VEC) {
        load8(src, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = 0.0f;
            if (i < n) {
                if constexpr (sizeof(T) == 4)
                    x[i] = src[i];
                else
                    x[i] = __uint_as_float(static_cast<uint32_t>(src[i]) << 16);
            }
        }
    }
}

// VEC: M is a multiple of 8, so that rows are aligned.
template <typename TI, typename TO, bool VEC>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(CombineParams p)
{
    const uint32_t piece = blockIdx.x * kCombineThreads + threadIdx.x;
    if (piece >= p.pieces) return;
    const uint32_t row = piece / p.per_row;
    const int64_t m = int64_t(piece - row * p.per_row.d) * 8;
    const int n = static_cast<int>(min(int64_t(8), p.M - m));
    const int32_t *slots = p.slots + int64_t(row) * p.top;
    const float *weights = p.weights + int64_t(row) * p.top;
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
    constexpr int U = 4;                              // rows under way together
    for (int j0 = 0; j0 < p.top; j0 += U) {
        float x[U][8], w[U];
        bool have[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = j0 + u < p.top;
            const int64_t slot = in ? slots[j0 + u] : -1;
            w[u] = in ? weights[j0 + u] : 0.0f;
            have[u] = slot >= 0 && slot < p.pairs;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[u][i] = 0.0f;
            if (have[u]) fetch8<VEC>(static_cast<const TI *>(p.y) + slot * p.M + m, n, x[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = fmaf(w[u], x[u][i], sum[i]);
    }
    TO *dst = static_cast<TO *>(p.out) + int64_t(row) * p.M + m;
    if constexpr (VEC) {
        store8(dst, sum);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) {
                if constexpr (sizeof(TO) == 4)
                    dst[i] = sum[i];
                else
                    dst[i] = static_cast<TO>(f32_to_bf16_bits(sum[i]));
            }
    }
}

}  // namespace qg
