// mx_few.hpp -- MX products for few rows: the weights are streamed once from
// memory straight into the operand registers.
//
// A wave takes MI blocks of 16 outputs (with SILU of the gate and of the up matrix)
// and up to 16 rows. KS waves share the same outputs, take runs of 512 inputs in
// turn, and their sums are added through LDS in a fixed order; a workgroup of four
// waves so takes 16 MI * 4 / KS outputs. A weight row's 64 bytes of a step are read
// by its four lanes, its scales of a run by one load of 16 bytes (asked for step by
// step, 4 bytes of each row, they cost a third of the time: 151936 x 2048, one row
// 49 us, 33 without any scales; now 30). The loop has no branches, so that
// the compiler knows how many loads are under way.
//
// Measured a call among others, e4m3 rows, on weights that come from memory (copies of them
// in turn) and in brackets on the same ones again, which the last cache holds in part.
// Bound by HBM where the weights are many: 151936 x 2048, one row, 33 us [30], 5.0 TB/s; 64
// x 8 rows of 128 experts, 1024 -> 2048, 30 us [27], 4.8 TB/s. 17408 x 5120 are 47 MB, 9 us
// of HBM: one row 17 us [12], 16 rows 23 [17]; there a launch, a wave's first loads and
// the sum of the waves are a large part, and with 16 rows as many bytes of rows as of
// weights, loaded and split for every 32 outputs anew. 6144 x 2048, one row, 6.5 us is the
// launch.
#pragma once

#include "mx_gemm.hpp"

namespace qg {

constexpr int kFewThreads = 256;
constexpr int kFewWaves = kFewThreads / 64;
constexpr int kFewRun = 512;        // inputs a wave takes at a time: four steps of 128, loaded in two halves

template <int XF, typename T, bool SILU, bool GROUPED, int MI, int KS>
__global__ __launch_bounds__(kFewThreads) void mx_few_kernel(MxGemmParams p)
{
    constexpr int WI = SILU ? 2 : 1, WB = MI * WI;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int tm = blockIdx.x % p.tiles_m, tn = blockIdx.x / p.tiles_m;
    int64_t r0, e = 0;
    int rows;
    if constexpr (GROUPED) {
        const GroupTile t = group_tile<16>(p.offsets, p.experts, p.N, tn);
        if (t.e < 0) return;
        e = t.e, r0 = t.r0, rows = t.r1 - t.r0;
    } else {
        r0 = int64_t(tn) * 16;
        rows = static_cast<int>(min(int64_t(16), p.N - r0));
    }
    const int64_t m0 = int64_t(tm) * (16 * MI * kFewWaves / KS) + 16 * MI * (wave / KS);
    const int outs = static_cast<int>(max(int64_t(0), min(int64_t(16 * MI), p.M - m0)));
    const int64_t wrb = p.K / 2, xrb = mx_bytes<XF>(p.K);

    __amdgpu_buffer_rsrc_t wbuf[WI], wsbuf[WI];
#pragma unroll
    for (int i = 0; i < WI; ++i) {
        const int64_t row = (e * WI + i) * p.M + min(m0, p.M - 1);
        wbuf[i] = mx_buffer(p.wc + row * wrb, outs * wrb);
        wsbuf[i] = mx_buffer(p.ws + row * p.pitch, int64_t(outs) * p.pitch);
    }
    const bool gather = GROUPED && p.order;
    const int64_t xfirst = gather ? 0 : r0, xin = gather ? p.x_rows : rows;
    const auto xbuf = mx_buffer(p.xc + xfirst * xrb, xin * xrb);
    const auto xsbuf = mx_buffer(p.xs + xfirst * p.pitch, xin * p.pitch);
    const int64_t xrow = x_row<GROUPED>(p, r0, rows, r);
    const uint32_t xoff = xrow < 0 ? kMxOut : static_cast<uint32_t>(xrow * xrb);
    const uint32_t xsoff = xrow < 0 ? kMxOut : static_cast<uint32_t>(xrow * p.pitch);
    const uint32_t woff = static_cast<uint32_t>(r * wrb), wsoff = static_cast<uint32_t>(r * p.pitch);

    constexpr int XP = kXParts<XF>;                  // 16-byte pieces of x a lane and step, and operands
    struct Scales {
        u32x4 w[WB], x;
    };
    const auto load_scales = [&](Scales &S, int run) {
#pragma unroll
        for (int i = 0; i < WB; ++i)
            S.w[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wsbuf[i % WI], wsoff + 16 * (i / WI) * p.pitch + run * (kFewRun / 32), 0, 0));
        S.x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xsbuf, xsoff + run * (kFewRun / 32), 0, 0));
    };
    struct Half {
        u32x4 w[WB][2], x[2][XP];
    };
    const auto load = [&](Half &H, int half) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k = half * (kFewRun / 2) + 128 * s;
#pragma unroll
            for (int h = 0; h < XP; ++h) {
                // inputs behind the row's end are zeros (the weights' there are any finite numbers)
                const int at = XF == kMxE2M1 ? k + 32 * g : k + 64 * h + 16 * g;
                const uint32_t off = mx_in_or_out(xoff + static_cast<uint32_t>(mx_bytes<XF>(at)), at, p.K);
                H.x[s][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xbuf, off, 0, 0));
            }
#pragma unroll
            for (int i = 0; i < WB; ++i)
                H.w[i][s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                          wbuf[i % WI], woff + 16 * (i / WI) * static_cast<uint32_t>(wrb) + k / 2 + 16 * g, 0, 0));
        }
    };
    f32x4 acc[WB];
#pragma unroll
    for (int i = 0; i < WB; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const auto multiply = [&](const Half &H, const Scales &S, int half, int first) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            // scales behind the row's end count as 2^-127
            const bool in = half * (kFewRun / 2) + 128 * s + 32 * g < p.K;
            i32x8 b[XP];
            x_operands<XF>(H.x[s][0], H.x[s][XP - 1], b);
            const int sb = in ? static_cast<int>(S.x[first + s] >> (8 * g)) : 0;
#pragma unroll
            for (int h = 0; h < XP; ++h)
#pragma unroll
                for (int i = 0; i < WB; ++i) {
                    const u32x4 w = H.w[i][s];
                    const i32x8 a = {int(w[0]), int(w[1]), int(w[2]), int(w[3]), 0, 0, 0, 0};
                    const int sa = in ? static_cast<int>(S.w[i][first + s] >> (8 * g)) : 0;
                    acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b[h], acc[i], kMxE2M1, XF, 0, sa, 0, sb);
                }
        }
    };
    const int runs = (p.K + kFewRun - 1) / kFewRun;
    int u = wave % KS;
    if (u < runs) {
        Scales S;
        Half A, B;
        load_scales(S, u);
        load(A, 2 * u);
        for (; u + KS < runs; u += KS) {
            Scales next;
            load(B, 2 * u + 1);
            load_scales(next, u + KS);
            __builtin_amdgcn_sched_barrier(0);
            multiply(A, S, 2 * u, 0);
            load(A, 2 * (u + KS));
            __builtin_amdgcn_sched_barrier(0);
            multiply(B, S, 2 * u + 1, 2);
            S = next;
        }
        if ((2 * u + 1) * (kFewRun / 2) < p.K) {
            load(B, 2 * u + 1);
            multiply(A, S, 2 * u, 0);
            multiply(B, S, 2 * u + 1, 2);
        } else {
            multiply(A, S, 2 * u, 0);
        }
    }
    T *y = static_cast<T *>(p.y);
    const auto value = [&](float v, float u) { return !SILU ? v : sizeof(T) == 4 ? silu_mul(v, u) : silu_mul_bf16(v, u); };
    const auto put = [&](T *dst, float v) {
        if constexpr (sizeof(T) == 4)
            *dst = v;
        else
            *dst = static_cast<T>(f32_to_bf16_bits(v));
    };
    if constexpr (KS == 1) {
        // column r is a row of x, element v of block i output 16 i + 4 g + v
        if (r < rows) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int m = 16 * i + 4 * g + v;
                    if (m < outs) put(y + (r0 + r) * p.M + m0 + m, value(acc[WI * i][v], acc[WI * i + WI - 1][v]));
                }
        }
    } else {
        __shared__ f32x4 sums[kFewWaves][WB][64];
#pragma unroll
        for (int i = 0; i < WB; ++i) sums[wave][i][lane] = acc[i];
        __syncthreads();
        // a thread of the KS waves: output t % 16 of row t / 16; it lies in lane (m / 4) * 16 + n, element m % 4
        const int first = wave / KS * KS;
#pragma unroll
        for (int t = lane + 64 * (wave % KS); t < 256; t += 64 * KS) {
            const int n = t >> 4, m = t & 15, at = (m >> 2) * 16 + n;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                float v[WI];
#pragma unroll
                for (int h = 0; h < WI; ++h) {
                    v[h] = 0.0f;
#pragma unroll
                    for (int w = 0; w < KS; ++w) v[h] += reinterpret_cast<const float *>(&sums[first + w][WI * i + h][at])[m & 3];
                }
                if (16 * i + m < outs && n < rows) put(y + (r0 + n) * p.M + m0 + 16 * i + m, value(v[0], v[WI - 1]));
            }
        }
    }
}

}  // namespace qg
