// mx_mid.hpp -- MX products for some tens of rows: the weights are streamed
// once from memory into the operand registers, the rows of x are shared by
// the workgroup's waves through LDS.
//
// A workgroup of four waves takes 32 MI weight rows and 16 NJ rows of x. Two waves
// lie side by side along the weights, with MI blocks of 16 rows each, and two
// split the inputs: of a stage of 256 inputs each takes one step of 128. x comes
// by loads that go to LDS directly, into a ring of D stages; a lane's weights are
// loaded AHEAD stages ahead. With SILU a wave's blocks are of the
// gate and of the up matrix in turn. The sums of the two waves are added through
// LDS in a fixed order.
#pragma once

#include "mx_tile.hpp"

namespace qg {

constexpr int kMidThreads = 256;
// stages whose weights are under way (of e4m3 a stage's products take twice as long)
template <int XF> constexpr int kMidAhead = XF == kMxE2M1 ? 2 : 1;

template <int XF, int MI, int NJ>
struct MxMidLds {
    static constexpr int D = XF == kMxE2M1 ? 4 : 3;
    static constexpr int xrow = static_cast<int>(mx_bytes<XF>(kTileK)), s = 16 * NJ * xrow, stage = s + 16 * NJ * kTileScale;
    static constexpr int sums = 4 * MI * (NJ / 2) * 1024;     // half of every wave's
    static constexpr int bytes = D * stage > sums ? D * stage : sums;
};

template <int XF, typename T, bool SILU, bool GROUPED, int MI, int NJ>
__global__ __launch_bounds__(kMidThreads, MI * NJ <= 24 ? 2 : 1) void mx_mid_kernel(MxGemmParams p)
{
    using L = MxMidLds<XF, MI, NJ>;
    constexpr int WI = SILU ? 2 : 1, OB = MI / WI, XP = kXParts<XF>, D = L::D, AHEAD = kMidAhead<XF>;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4, half = wave & 1, side = wave >> 1;
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
    const int64_t m0 = int64_t(tm) * (32 * OB) + 16 * OB * side;        // this wave's first output
    const int outs = static_cast<int>(max(int64_t(0), min(int64_t(16 * OB), p.M - m0)));
    const int wrb = p.K / 2, xrb = static_cast<int>(mx_bytes<XF>(p.K));

    __amdgpu_buffer_rsrc_t wbuf[WI], wsbuf[WI];
#pragma unroll
    for (int i = 0; i < WI; ++i) {
        const int64_t row = (e * WI + i) * p.M + min(m0, p.M - 1);
        wbuf[i] = mx_buffer(p.wc + row * wrb, int64_t(outs) * wrb);
        wsbuf[i] = mx_buffer(p.ws + row * p.pitch, int64_t(outs) * p.pitch);
    }
    const bool gather = GROUPED && p.order;
    const int64_t xfirst = gather ? 0 : r0, xin = gather ? p.x_rows : rows;
    const auto xbuf = mx_buffer(p.xc + xfirst * xrb, xin * xrb);
    const auto xsbuf = mx_buffer(p.xs + xfirst * p.pitch, xin * p.pitch);

    // what this lane brings to LDS: pieces of rows of x, and of 32 rows' scales 4 bytes
    constexpr int XC = L::xrow / 16, XR = 64 / XC, XN = 16 * NJ / XR, XL = (XN + 3) / 4;      // loads of a stage, and of a wave
    uint32_t xoff[XL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        const int row = XR * min(i * 4 + wave, XN - 1) + lane / XC;      // (every wave has as many: the last may come twice)
        const int64_t x = x_row<GROUPED>(p, r0, rows, row);
        xoff[i] = x < 0 ? kMxOut : static_cast<uint32_t>(x * xrb + 16 * ((lane % XC) ^ mx_swizzle<XC>(row)));
    }
    constexpr int SN = NJ / 2;
    static_assert(SN <= 4, "a load of scales a wave");
    const int sq = wave % SN;                        // (two waves may have the same)
    const int64_t srow = x_row<GROUPED>(p, r0, rows, 32 * sq + lane / 2);
    const uint32_t soff = srow < 0 ? kMxOut : static_cast<uint32_t>(srow * p.pitch + 4 * (lane & 1));
    const int stages = (p.K + kTileK - 1) / kTileK;
    const auto fill = [&](int t) {
        uint8_t *dst = lds + t % D * L::stage;
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int q = min(i * 4 + wave, XN - 1), row = XR * q + lane / XC;
            // inputs behind the row's end are zeros (the weights' there are any finite numbers)
            const int k = t * kTileK + ((lane % XC) ^ mx_swizzle<XC>(row)) * (XF == kMxE2M1 ? 32 : 16);
            mx_to_lds16(xbuf, dst + q * 1024, mx_in_or_out(xoff[i] + t * L::xrow, k, p.K));
        }
        mx_to_lds4(xsbuf, dst + L::s + sq * 256, soff + t * kTileScale);
    };
    struct Regs {
        u32x4 w[MI];
        uint32_t sw[MI];
    };
    const uint32_t woff = static_cast<uint32_t>(r * wrb + 16 * g), wsoff = static_cast<uint32_t>(r * p.pitch);
    const auto load = [&](Regs &R, int t) {
        const int k = t * kTileK + 128 * half;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int by = 16 * (i / WI);
            R.w[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wbuf[i % WI], woff + by * wrb + k / 2, 0, 0));
            R.sw[i] = __builtin_amdgcn_raw_buffer_load_b32(wsbuf[i % WI], wsoff + by * p.pitch + k / 32, 0, 0);
        }
    };
    f32x4 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const auto multiply = [&](const Regs &R, int t) {
        const uint8_t *src = lds + t % D * L::stage;
        // scales behind the row's end count as 2^-127
        const bool in = t * kTileK + 128 * half + 32 * g < p.K;
        int sw[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) sw[i] = in ? static_cast<int>(R.sw[i] >> (8 * g)) : 0;
        // a block's rows are read while those of the one before are multiplied
        u32x4 lo[2], hi[2];
        int sx[2];
        const auto read = [&](int j) {
            const uint8_t *row = src + (16 * j + r) * L::xrow;
            if constexpr (XF == kMxE2M1) {
                lo[j & 1] = hi[j & 1] = *reinterpret_cast<const u32x4 *>(row + 16 * ((4 * half + g) ^ mx_swizzle<XC>(r)));
            } else {
                lo[j & 1] = *reinterpret_cast<const u32x4 *>(row + 16 * ((8 * half + g) ^ mx_swizzle<XC>(r)));
                hi[j & 1] = *reinterpret_cast<const u32x4 *>(row + 16 * ((8 * half + 4 + g) ^ mx_swizzle<XC>(r)));
            }
            sx[j & 1] = *reinterpret_cast<const int *>(src + L::s + (16 * j + r) * kTileScale + 4 * half);
        };
        read(0);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            __builtin_amdgcn_sched_barrier(0);
            if (j + 1 < NJ) read(j + 1);
            i32x8 b[XP];
            x_operands<XF>(lo[j & 1], hi[j & 1], b);
            const int s = in ? sx[j & 1] >> (8 * g) : 0;
#pragma unroll
            for (int h = 0; h < XP; ++h)
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const i32x8 a = {int(R.w[i][0]), int(R.w[i][1]), int(R.w[i][2]), int(R.w[i][3]), 0, 0, 0, 0};
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b[h], acc[i][j], kMxE2M1, XF, 0, sw[i], 0, s);
                }
        }
    };

    // Stage t's x was asked for D - 1 stages before it and has come once all but
    // the memory operations since are done; loads past the end read zeros. The loop
    // has no branches, so that the compiler knows how many loads are under way.
    constexpr int WL = 2 * MI, FL = XL + 1;          // a wave's loads of a stage, to registers and to LDS
    Regs R[AHEAD + 1];
    for (int t = 0; t < D - 1; ++t) fill(t);
#pragma unroll
    for (int t = 0; t < AHEAD; ++t) load(R[t], t);
    mx_meet<(D - 2) * FL + AHEAD * WL>();
    const auto stage = [&](int t, int u) {
        mx_meet<WL + (D - 2) * (FL + WL)>();
        fill(t + D - 1);
        load(R[(u + AHEAD) % (AHEAD + 1)], t + AHEAD);
        __builtin_amdgcn_sched_barrier(0);
        multiply(R[u], t);
    };
    int t = 0;
    for (; t + AHEAD < stages; t += AHEAD + 1) {
#pragma unroll
        for (int u = 0; u <= AHEAD; ++u) stage(t + u, u);
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
        if (t + u < stages) stage(t + u, u);
    mx_meet<0>();                                    // nobody reads x any more, and no load to LDS is under way

    // of the rows' blocks each wave finishes half, with the other's sums of them
    constexpr int HJ = NJ / 2;
    f32x4 *sums = reinterpret_cast<f32x4 *>(lds);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < HJ; ++j) {
            f32x4 v;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = half ? acc[i][j][q] : acc[i][HJ + j][q];
            sums[((wave * MI + i) * HJ + j) * 64 + lane] = v;
        }
    __syncthreads();
    T *y = static_cast<T *>(p.y) + r0 * p.M + m0;
#pragma unroll
    for (int j = 0; j < HJ; ++j) {
        const int n = 16 * (half ? HJ + j : j) + r;
#pragma unroll
        for (int i = 0; i < MI; i += WI) {
            f32x4 v[WI];
#pragma unroll
            for (int h = 0; h < WI; ++h) {
                const f32x4 other = sums[(((wave ^ 1) * MI + i + h) * HJ + j) * 64 + lane];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[h][q] = (half ? acc[i + h][HJ + j][q] : acc[i + h][j][q]) + other[q];
            }
            const int m = 16 * (i / WI) + 4 * g;
            float out[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                out[q] = !SILU ? v[0][q] : sizeof(T) == 4 ? silu_mul(v[0][q], v[WI - 1][q]) : silu_mul_bf16(v[0][q], v[WI - 1][q]);
            T *dst = y + n * p.M + m;
            if (n < rows && m < outs) {
                if (p.M % 4 == 0) {
                    if constexpr (sizeof(T) == 4)
                        *reinterpret_cast<f32x4 *>(dst) = f32x4{out[0], out[1], out[2], out[3]};
                    else
                        *reinterpret_cast<u32x2 *>(dst) = u32x2{f32_to_bf16_pair(out[0], out[1]), f32_to_bf16_pair(out[2], out[3])};
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (m + q < outs) {
                            if constexpr (sizeof(T) == 4)
                                dst[q] = out[q];
                            else
                                dst[q] = static_cast<T>(f32_to_bf16_bits(out[q]));
                        }
                }
            }
        }
    }
}

}  // namespace qg
