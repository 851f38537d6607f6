// mx_few.hpp -- MX products for few rows: the weights are streamed once from
// memory straight into the operand registers.
//
// A workgroup takes 16 outputs and up to 16 NJ rows; its four waves take
// runs of 256 inputs in turn and their sums are added through LDS in a fixed
// order. A weight row's 64 bytes of a step are read by its four lanes.
#pragma once

#include "mx_gemm.hpp"

namespace qg {

constexpr int kFewThreads = 256;
constexpr int kFewWaves = kFewThreads / 64;
constexpr int kFewChunk = 256;      // inputs a wave takes at a time: two steps of 128

template <int XF, typename T, bool SILU, bool GROUPED, int NJ>
__global__ __launch_bounds__(kFewThreads) void mx_few_kernel(MxGemmParams p)
{
    constexpr int WI = SILU ? 2 : 1;
    __shared__ f32x4 sums[kFewWaves][WI * NJ][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int tm = blockIdx.x % p.tiles_m, tn = blockIdx.x / p.tiles_m;
    int64_t r0, e = 0;
    int rows;
    if constexpr (GROUPED) {
        const GroupTile t = group_tile<16 * NJ>(p.offsets, p.experts, p.N, tn);
        if (t.e < 0) return;
        e = t.e, r0 = t.r0, rows = t.r1 - t.r0;
    } else {
        r0 = int64_t(tn) * (16 * NJ);
        rows = static_cast<int>(min(int64_t(16 * NJ), p.N - r0));
    }
    const int64_t m0 = int64_t(tm) * 16;
    const int outs = static_cast<int>(min(int64_t(16), p.M - m0));
    const int64_t wrb = p.K / 2, xrb = mx_bytes<XF>(p.K);

    __amdgpu_buffer_rsrc_t wbuf[WI], wsbuf[WI];
#pragma unroll
    for (int i = 0; i < WI; ++i) {
        const int64_t row = (e * WI + i) * p.M + m0;
        wbuf[i] = mx_buffer(p.wc + row * wrb, outs * wrb);
        wsbuf[i] = mx_buffer(p.ws + row * p.pitch, int64_t(outs) * p.pitch);
    }
    const bool gather = GROUPED && p.order;
    const int64_t xfirst = gather ? 0 : r0, xin = gather ? p.x_rows : rows;
    const auto xbuf = mx_buffer(p.xc + xfirst * xrb, xin * xrb);
    const auto xsbuf = mx_buffer(p.xs + xfirst * p.pitch, xin * p.pitch);
    uint32_t xoff[NJ], xsoff[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int64_t row = x_row<GROUPED>(p, r0, rows, 16 * j + r);
        xoff[j] = row < 0 ? kMxOut : static_cast<uint32_t>(row * xrb);
        xsoff[j] = row < 0 ? kMxOut : static_cast<uint32_t>(row * p.pitch);
    }
    const uint32_t woff = static_cast<uint32_t>(r * wrb), wsoff = static_cast<uint32_t>(r * p.pitch);

    constexpr int XP = kXParts<XF>;                  // 16-byte pieces of x a lane and step, and operands
    struct Regs {
        u32x4 w[WI][2], x[NJ][2][XP];
        uint32_t sw[WI][2], sx[NJ][2];
    };
    const auto load = [&](Regs &R, int c) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k = c * kFewChunk + 128 * s;
#pragma unroll
            for (int i = 0; i < WI; ++i) {
                R.w[i][s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wbuf[i], woff + k / 2 + 16 * g, 0, 0));
                R.sw[i][s] = __builtin_amdgcn_raw_buffer_load_b32(wsbuf[i], wsoff + k / 32, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
#pragma unroll
                for (int h = 0; h < XP; ++h) {
                    // inputs behind the row's end are zeros (the weights' there are any finite numbers)
                    const int at = XF == kMxE2M1 ? k + 32 * g : k + 64 * h + 16 * g;
                    const uint32_t off = mx_in_or_out(xoff[j] + static_cast<uint32_t>(mx_bytes<XF>(at)), at, p.K);
                    R.x[j][s][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xbuf, off, 0, 0));
                }
                R.sx[j][s] = __builtin_amdgcn_raw_buffer_load_b32(xsbuf, xsoff[j] + k / 32, 0, 0);
            }
        }
    };
    f32x4 acc[WI][NJ];
#pragma unroll
    for (int i = 0; i < WI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const auto multiply = [&](const Regs &R, int c) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            // scales behind the row's end count as 2^-127
            const bool in = c * kFewChunk + 128 * s + 32 * g < p.K;
            i32x8 b[NJ][XP];
            int sb[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                x_operands<XF>(R.x[j][s][0], R.x[j][s][XP - 1], b[j]);
                sb[j] = in ? static_cast<int>(R.sx[j][s] >> (8 * g)) : 0;
            }
#pragma unroll
            for (int i = 0; i < WI; ++i) {
                const u32x4 w = R.w[i][s];
                const i32x8 a = {int(w[0]), int(w[1]), int(w[2]), int(w[3]), 0, 0, 0, 0};
                const int sa = in ? static_cast<int>(R.sw[i][s] >> (8 * g)) : 0;
#pragma unroll
                for (int h = 0; h < XP; ++h)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b[j][h], acc[i][j], kMxE2M1, XF, 0, sa, 0, sb[j]);
            }
        }
    };
    const int chunks = (p.K + kFewChunk - 1) / kFewChunk;
    int c = wave;
    if (c < chunks) {
        Regs A, B;
        load(A, c);
        for (;;) {
            // loads of the chunk after are under way while this one is multiplied
            // (behind the last, offsets in a valid range or out of it: never used)
            const int n = c + kFewWaves;
            if (n < chunks) load(B, n);
            multiply(A, c);
            if (n >= chunks) break;
            const int n2 = n + kFewWaves;
            if (n2 < chunks) load(A, n2);
            multiply(B, n);
            if (n2 >= chunks) break;
            c = n2;
        }
    }
#pragma unroll
    for (int i = 0; i < WI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) sums[wave][i * NJ + j][lane] = acc[i][j];
    __syncthreads();
    // thread t: output t % 16 of row t / 16; it lies in lane (m / 4) * 16 + n, element m % 4
    const int n = threadIdx.x >> 4, m = threadIdx.x & 15;
    const int at = (m >> 2) * 16 + n;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        float v[WI];
#pragma unroll
        for (int i = 0; i < WI; ++i) {
            v[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w) v[i] += reinterpret_cast<const float *>(&sums[w][i * NJ + j][at])[m & 3];
        }
        const float out = !SILU ? v[0] : sizeof(T) == 4 ? silu_mul(v[0], v[WI - 1]) : silu_mul_bf16(v[0], v[WI - 1]);
        if (m < outs && 16 * j + n < rows) {
            T *dst = static_cast<T *>(p.y) + (r0 + 16 * j + n) * p.M + m0 + m;
            if constexpr (sizeof(T) == 4)
                *dst = out;
            else
                *dst = static_cast<T>(f32_to_bf16_bits(out));
        }
    }
}

}  // namespace qg
