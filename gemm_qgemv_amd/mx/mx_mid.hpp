// mx_mid.hpp -- MX products for some tens of rows: the weights are streamed
// once from memory into the operand registers, the rows of x are shared by
// the workgroup's waves through LDS.
//
// A workgroup takes 32 MI weight rows and 16 NJ rows of x. Of its four waves two lie
// side by side along the weights, with MI blocks of 16 rows each, and two split the
// inputs into parts, of which each takes a step of 128 a stage. x comes by loads
// that go to LDS directly, into a ring of D stages; a lane's weights are loaded
// a stage ahead, their scales two stages at a time. With SILU a wave's blocks
// are of the gate and of the up matrix in turn. The parts' sums are added through
// LDS in a fixed order.
//
// Two parts of two waves, so that a compute unit has room for two workgroups of most
// sizes, whose loads and products overlap where there are as many (77 x 2 x 17408 x 5120,
// e4m3, has 272 workgroups, so that most units hold one: 58 us, with four parts 72).
// Bound by the loads' latency: weights are asked for one stage ahead, 16 KiB of them
// a compute unit and workgroup, and a stage takes as long as they do (matrix and vector
// instructions issue a fifth of the time each). 17408 x 5120 x 90 rows e2m1 22 us, 28
// with weights that come from memory (1.7 TB/s of them), x 60 e4m3 32 and 34.
#pragma once

#include <type_traits>

#include "mx_tile.hpp"

namespace qg {

constexpr int kMidParts = 2, kMidThreads = 64 * 2 * kMidParts;
constexpr int kMidK = 128;       // inputs of a part and stage

template <int XF, int MI, int NJ>
struct MxMidLds {
    static constexpr int D = 3;
    static constexpr int xrow = static_cast<int>(mx_bytes<XF>(kMidK)), s = 16 * NJ * xrow;
    static constexpr int sn = (NJ + 3) / 4, part = s + sn * 256, stage = kMidParts * part;     // loads of 64 rows' scales
    static constexpr int sums = 4 * (MI * NJ / 2) * 1024;      // half of the blocks of four waves
    static constexpr int bytes = D * stage > sums ? D * stage : sums;
};

// A wave's memory operations since it asked for the x of the stage at place u of
// four: a stage asks for x (FL loads) and MI weights, one in two for MI scales. They
// come in order, so that the wait holds only if a stage asks for x first, whatever
// the compiler's scheduler does: mx_x_first stands behind it.
template <int MI, int FL, int D>
__host__ __device__ constexpr int mx_mid_since(int u)
{
    int n = 0;
    for (int s = u + 8 - D + 1; s < u + 8; ++s) n += MI + (s % 2 == 0 ? MI : 0) + (s > u + 8 - D + 1 ? FL : 0);
    return n;
}

__device__ __forceinline__ void mx_x_first() { __builtin_amdgcn_sched_barrier(0); }

template <int XF, typename T, bool SILU, bool GROUPED, int MI, int NJ>
__global__ __launch_bounds__(kMidThreads, 2) void mx_mid_kernel(MxGemmParams p)
{
    using L = MxMidLds<XF, MI, NJ>;
    constexpr int WI = SILU ? 2 : 1, OB = MI / WI, XP = kXParts<XF>, D = L::D;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4, part = wave % kMidParts, side = wave / kMidParts;
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

    // this wave's inputs: k0 .. k1 - 1, in stages of 128
    const int each = ((p.K + kMidParts - 1) / kMidParts + kMidK - 1) / kMidK * kMidK, stages = each / kMidK;
    const int k0 = part * each, k1 = min(p.K, k0 + each);
    // what this lane brings to LDS of its part's x (the other side's wave brings the
    // other half): pieces of rows, and 4 bytes of a row's scales
    constexpr int XC = L::xrow / 16, XR = 64 / XC, XN = 16 * NJ / XR, XL = (XN + 1) / 2;      // loads of a stage, and of a wave
    uint32_t xoff[XL];
    int xq[XL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        xq[i] = min(i * 2 + side, XN - 1);           // (both waves have as many: the last may come twice)
        const int row = XR * xq[i] + lane / XC;
        const int64_t x = x_row<GROUPED>(p, r0, rows, row);
        xoff[i] = x < 0 ? kMxOut : static_cast<uint32_t>(x * xrb + mx_bytes<XF>(k0) + 16 * ((lane % XC) ^ mx_swizzle<XC>(row)));
    }
    const int sq = min(side, L::sn - 1);
    const int64_t srow = x_row<GROUPED>(p, r0, rows, 64 * sq + lane);
    const uint32_t soff = srow < 0 ? kMxOut : static_cast<uint32_t>(srow * p.pitch + k0 / kMxBlock);
    const auto fill = [&](int t) __attribute__((always_inline)) {
        uint8_t *dst = lds + t % D * L::stage + part * L::part;
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            // inputs behind the row's end are zeros (the weights' there are any finite
            // numbers), and what is behind the part's is not asked for
            const int k = k0 + t * kMidK + ((lane % XC) ^ mx_swizzle<XC>(XR * xq[i] + lane / XC)) * (XF == kMxE2M1 ? 32 : 16);
            mx_to_lds16(xbuf, dst + xq[i] * 1024, mx_in_or_out(xoff[i] + t * L::xrow, k, k1));
        }
        mx_to_lds4(xsbuf, dst + L::s + sq * 256, soff + t * (kMidK / kMxBlock));
    };
    // a lane's weights of a stage, and its scales of two
    struct Weights {
        u32x4 w[MI];
    };
    struct Scales {
        u32x2 w[MI];
    };
    const uint32_t woff = static_cast<uint32_t>(r * wrb + k0 / 2 + 16 * g), wsoff = static_cast<uint32_t>(r * p.pitch + k0 / kMxBlock);
    const auto load = [&](Weights &R, int t) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
            R.w[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wbuf[i % WI], woff + 16 * (i / WI) * wrb + t * (kMidK / 2), 0, 0));
    };
    const auto load_scales = [&](Scales &S, int two) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
            S.w[i] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(wsbuf[i % WI], wsoff + 16 * (i / WI) * p.pitch + two * 8, 0, 0));
    };
    f32x4 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const auto multiply = [&](const Weights &R, const Scales &S, int t, int u) __attribute__((always_inline)) {
        const uint8_t *src = lds + t % D * L::stage + part * L::part;
        // scales behind the row's end count as 2^-127
        const bool in = k0 + t * kMidK + 32 * g < p.K;
        int sw[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) sw[i] = in ? static_cast<int>(S.w[i][u % 2] >> (8 * g)) : 0;
        // Blocks of 16 rows in turn: the next one's rows are read while one is multiplied
        // (the other wave of a SIMD fills the matrix cores while operands are made).
        u32x4 lo[2], hi[2];
        int raw[2];
        const auto read = [&](int j) {
            const uint8_t *row = src + (16 * j + r) * L::xrow;
            lo[j & 1] = hi[j & 1] = *reinterpret_cast<const u32x4 *>(row + 16 * (g ^ mx_swizzle<XC>(r)));
            if constexpr (XF != kMxE2M1) hi[j & 1] = *reinterpret_cast<const u32x4 *>(row + 16 * ((4 + g) ^ mx_swizzle<XC>(r)));
            raw[j & 1] = *reinterpret_cast<const int *>(src + L::s + (16 * j + r) * 4);
        };
        read(0);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            __builtin_amdgcn_sched_barrier(0);
            if (j + 1 < NJ) read(j + 1);
            i32x8 b[XP];
            x_operands<XF>(lo[j & 1], hi[j & 1], b);
            const int sx = in ? raw[j & 1] >> (8 * g) : 0;
#pragma unroll
            for (int h = 0; h < XP; ++h)
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const i32x8 a = {int(R.w[i][0]), int(R.w[i][1]), int(R.w[i][2]), int(R.w[i][3]), 0, 0, 0, 0};
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b[h], acc[i][j], kMxE2M1, XF, 0, sw[i], 0, sx);
                }
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    // Stage t's x was asked for D - 1 stages before it and has come once all but
    // the memory operations since are done; loads past the end read zeros. The loop
    // has no branches, so that the compiler knows how many loads are under way.
    constexpr int FL = XL + 1;
    Weights R[2];
    Scales S[2];
    for (int t = 0; t < D - 1; ++t) fill(t);
    mx_x_first();
    load(R[0], 0);
    load_scales(S[0], 0);
    mx_meet<(D - 2) * FL + MI * 2>();
    const auto stage = [&](int t, auto place) __attribute__((always_inline)) {
        constexpr int u = decltype(place)::value;    // t % 4
        mx_meet<mx_mid_since<MI, FL, D>(u)>();
        fill(t + D - 1);
        mx_x_first();
        load(R[u % 2 ^ 1], t + 1);
        if constexpr (u % 2 == 0) load_scales(S[u / 2 ^ 1], t / 2 + 1);
        __builtin_amdgcn_sched_barrier(0);
        multiply(R[u % 2], S[u / 2], t, u);
    };
    constexpr std::integral_constant<int, 0> first{};
    constexpr std::integral_constant<int, 1> second{};
    constexpr std::integral_constant<int, 2> third{};
    constexpr std::integral_constant<int, 3> fourth{};
    int t = 0;
    for (; t + 4 <= stages; t += 4) {
        stage(t, first);
        stage(t + 1, second);
        stage(t + 2, third);
        stage(t + 3, fourth);
    }
    if (t < stages) stage(t, first);
    if (t + 1 < stages) stage(t + 1, second);
    if (t + 2 < stages) stage(t + 2, third);
    mx_meet<0>();                                    // nobody reads x any more, and no load to LDS is under way

    // Each part's wave finishes half of the blocks, with the other's sums of them: half
    // of the rows, or half of the outputs.
    f32x4 *sums = reinterpret_cast<f32x4 *>(lds);
    const int half = part, pair = side * 2 + half;
    constexpr bool BY_ROWS = NJ % 2 == 0;
    static_assert(BY_ROWS || MI % (2 * WI) == 0, "halves");
    constexpr int HI = BY_ROWS ? MI : MI / 2, HJ = BY_ROWS ? NJ / 2 : NJ;      // blocks of a half
    constexpr int DI = MI - HI, DJ = NJ - HJ;                                  // from the first half's to the second's
#pragma unroll
    for (int i = 0; i < HI; ++i)
#pragma unroll
        for (int j = 0; j < HJ; ++j) {
            f32x4 v;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = half ? acc[i][j][q] : acc[DI + i][DJ + j][q];
            sums[((pair * HI + i) * HJ + j) * 64 + lane] = v;
        }
    __syncthreads();
    T *y = static_cast<T *>(p.y) + r0 * p.M + m0;
#pragma unroll
    for (int j = 0; j < HJ; ++j) {
        const int n = 16 * (half ? DJ + j : j) + r;
#pragma unroll
        for (int i = 0; i < HI; i += WI) {
            f32x4 v[WI];
#pragma unroll
            for (int h = 0; h < WI; ++h) {
                const f32x4 other = sums[(((pair ^ 1) * HI + i + h) * HJ + j) * 64 + lane];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[h][q] = (half ? acc[DI + i + h][DJ + j][q] : acc[i + h][j][q]) + other[q];
            }
            const int m = 16 * ((half ? DI + i : i) / WI) + 4 * g;
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
