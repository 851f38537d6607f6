// mx_tile.hpp -- MX products for many rows: tiles of weights and activations
// brought from memory straight into LDS.
//
// A workgroup of WM x WN waves takes BM weight rows and BN rows of x; a stage
// is 256 inputs of both, with their scales, in one of two LDS buffers, filled
// by loads that go to LDS directly while the other is multiplied. A wave takes
// BM / WM x BN / WN of the tile in blocks of 32 x 32.
//
// Which inputs an instruction takes together is free as long as both operands
// agree: of the stage's 8 blocks a lane with g = 0 takes blocks 0..3 in turn, one
// with g = 1 blocks 4..7. So its scales of the whole stage are the four bytes
// of one dword, and the instruction's byte selector walks them.
//
// With SILU the tile's weight rows are 32 of the gate and 32 of the up matrix
// in turn, so that a lane holds both numbers of an output.
#pragma once

#include "mx_gemm.hpp"

namespace qg {

constexpr int kTileK = 256;      // inputs of a stage

template <int XF, int BM, int BN>
struct MxTileLds {
    static constexpr int wrow = kTileK / 2, xrow = static_cast<int>(mx_bytes<XF>(kTileK)), srow = kTileK / 32;
    static constexpr int x = BM * wrow, s = x + BN * xrow, stage = s + (BM + BN) * srow;
    static constexpr int bytes = 2 * stage;
};

// 16-byte chunk c of LDS row r lies at chunk c ^ swizzle(r): 16 lanes that
// read one chunk of 16 rows, or 8 of 8, meet no bank twice.
template <int CHUNKS>
__device__ __forceinline__ int mx_swizzle(int r)
{
    return CHUNKS == 16 ? r & 15 : (r & 7) ^ ((r >> 3) & 1);
}

template <int S, int XF, int TI, int TJ>
__device__ __forceinline__ void mx_tile_step(const uint8_t *wl, const uint8_t *xl, const int (&sw)[TI], const int (&sx)[TJ],
                                             f32x16 (&acc)[TI][TJ], int r, int g)
{
    constexpr int wrow = kTileK / 2, xrow = static_cast<int>(mx_bytes<XF>(kTileK));
    // (the swizzle goes by a row's low four bits, which r has)
    constexpr int XP = kXParts<XF>;
    i32x8 a[TI], b[TJ][XP];
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        const int row = 32 * i + r;
        const u32x4 v = *reinterpret_cast<const u32x4 *>(wl + row * wrow + 16 * ((4 * g + S) ^ mx_swizzle<8>(row)));
        a[i] = i32x8{int(v[0]), int(v[1]), int(v[2]), int(v[3]), 0, 0, 0, 0};
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
        const int row = 32 * j + r;
        if constexpr (XF == kMxE2M1) {
            const u32x4 v = *reinterpret_cast<const u32x4 *>(xl + row * xrow + 16 * ((4 * g + S) ^ mx_swizzle<8>(row)));
            x_operands<XF>(v, v, b[j]);
        } else {
            // bytes 0..15: half g of block S; bytes 16..31: half g of block 4 + S
            const u32x4 u = *reinterpret_cast<const u32x4 *>(xl + row * xrow + 16 * ((2 * S + g) ^ mx_swizzle<16>(row)));
            const u32x4 v = *reinterpret_cast<const u32x4 *>(xl + row * xrow + 16 * ((8 + 2 * S + g) ^ mx_swizzle<16>(row)));
            x_operands<XF>(u, v, b[j]);
        }
    }
#pragma unroll
    for (int h = 0; h < XP; ++h)
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int j = 0; j < TJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[i], b[j][h], acc[i][j], kMxE2M1, XF, S, sw[i], S, sx[j]);
}

template <int XF, typename T, bool SILU, bool GROUPED, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM *WN) void mx_tile_kernel(MxGemmParams p)
{
    using L = MxTileLds<XF, BM, BN>;
    constexpr int NW = WM * WN, TI = BM / WM / 32, TJ = BN / WN / 32, WI = SILU ? 2 : 1;
    static_assert(TI % WI == 0, "a wave holds gate and up rows of an output");
    extern __shared__ __align__(16) uint8_t lds[];

    // consecutive workgroups go to the 8 XCDs in turn: each XCD gets a run of
    // tiles, outputs first, which share rows of x in its L2
    const int ntiles = p.tiles_m * p.tiles_n;
    int bid = blockIdx.x;
    {
        const int each = ntiles >> 3, over = ntiles & 7, xcd = bid & 7, nth = bid >> 3;
        bid = xcd * each + min(xcd, over) + nth;
    }
    const int tm = bid % p.tiles_m, tn = bid / p.tiles_m;
    int64_t r0, e = 0;
    int rows;
    if constexpr (GROUPED) {
        const GroupTile t = group_tile<BN>(p.offsets, p.experts, p.N, tn);
        if (t.e < 0) return;
        e = t.e, r0 = t.r0, rows = t.r1 - t.r0;
    } else {
        r0 = int64_t(tn) * BN;
        rows = static_cast<int>(min(int64_t(BN), p.N - r0));
    }
    constexpr int OUTS = BM / WI;                    // outputs of a tile
    const int64_t m0 = int64_t(tm) * OUTS;
    const int outs = static_cast<int>(min(int64_t(OUTS), p.M - m0));
    const int64_t wrb = p.K / 2, xrb = mx_bytes<XF>(p.K);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, g = lane >> 5;

    const bool gather = GROUPED && p.order;
    const int64_t xfirst = gather ? 0 : r0, xin = gather ? p.x_rows : rows;
    const uint8_t *wbase[WI], *wsbase[WI];
#pragma unroll
    for (int i = 0; i < WI; ++i) {
        const int64_t row = (e * WI + i) * p.M + m0;
        wbase[i] = p.wc + row * wrb;
        wsbase[i] = p.ws + row * p.pitch;
    }
    const uint8_t *xbase = p.xc + xfirst * xrb, *xsbase = p.xs + xfirst * p.pitch;
    const int64_t wlen = outs * wrb, wslen = int64_t(outs) * p.pitch, xlen = xin * xrb, xslen = xin * p.pitch;

    // this lane's pieces of a stage. Weights: load i of the wave fills LDS rows 8 q .. 8 q + 7, q = i * NW + wave
    constexpr int WL = BM / 8 / NW, XR = 1024 / L::xrow, XL = BN / XR / NW, XC = L::xrow / 16;
    constexpr int SB = (BM + BN) / 32, SL = (SB + NW - 1) / NW;
    static_assert(WL * NW * 8 == BM && XL * NW * XR == BN, "whole loads");
    uint32_t woff[WL], xoff[XL], soff[SL];
    int xk[XL];                                      // first input of the x piece within the stage
#pragma unroll
    for (int i = 0; i < WL; ++i) {
        const int row = 8 * (i * NW + wave) + (lane >> 3);
        const int real = SILU ? (row >> 6) * 32 + (row & 31) : row;
        woff[i] = static_cast<uint32_t>(real * wrb + 16 * ((lane & 7) ^ mx_swizzle<8>(row)));
    }
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        const int row = XR * (i * NW + wave) + lane / XC, chunk = (lane % XC) ^ mx_swizzle<XC>(row);
        const int64_t at = x_row<GROUPED>(p, r0, rows, row);
        xoff[i] = at < 0 ? kMxOut : static_cast<uint32_t>(at * xrb + 16 * chunk);
        xk[i] = chunk * (XF == kMxE2M1 ? 32 : 16);
    }
#pragma unroll
    for (int i = 0; i < SL; ++i) {
        const int q = i * NW + wave, row = 32 * q + (lane >> 1);     // blocks of 32 rows, the weights' first
        if (row < BM) {
            soff[i] = static_cast<uint32_t>((SILU ? (row >> 6) * 32 + (row & 31) : row) * p.pitch + 4 * (lane & 1));
        } else {
            const int64_t at = row < BM + BN ? x_row<GROUPED>(p, r0, rows, row - BM) : -1;
            soff[i] = at < 0 ? kMxOut : static_cast<uint32_t>(at * p.pitch + 4 * (lane & 1));
        }
    }
    const int stages = (p.K + kTileK - 1) / kTileK;

    const auto fill = [&](int t, uint8_t *dst) {
        const int64_t wk = int64_t(t) * L::wrow, xk0 = int64_t(t) * L::xrow, sk = int64_t(t) * L::srow;
        const bool tail = (t + 1) * kTileK > p.K;
#pragma unroll
        for (int i = 0; i < WL; ++i) {
            const int q = i * NW + wave, part = SILU ? (q >> 2) & 1 : 0;
            const auto buf = mx_buffer(wbase[part] + wk, wlen - wk);
            mx_to_lds16(buf, dst + q * 1024, woff[i]);
        }
        const auto xbuf = mx_buffer(xbase + xk0, xlen - xk0);
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            // inputs behind the row's end are zeros (the weights' there are any finite numbers)
            const uint32_t off = tail && t * kTileK + xk[i] >= p.K ? kMxOut : xoff[i];
            mx_to_lds16(xbuf, dst + L::x + (i * NW + wave) * 1024, off);
        }
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            const int q = i * NW + wave;
            if (SL * NW != SB && q >= SB) break;
            const bool ofw = 32 * q < BM;
            const int part = SILU ? q & 1 : 0;
            const auto buf = mx_buffer((ofw ? wsbase[part] : xsbase) + sk, (ofw ? wslen : xslen) - sk);
            mx_to_lds4(buf, dst + L::s + q * 256, soff[i]);
        }
    };

    f32x16 acc[TI][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);

    const auto multiply = [&](int t, const uint8_t *src) {
        // scale bytes behind the row's end count as 2^-127
        const int left = p.K / 32 - t * (kTileK / 32) - 4 * g;
        const uint32_t mask = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1;
        int sw[TI], sx[TJ];
#pragma unroll
        for (int i = 0; i < TI; ++i)
            sw[i] = static_cast<int>(*reinterpret_cast<const uint32_t *>(src + L::s + (wm + 32 * i + r) * L::srow + 4 * g) & mask);
#pragma unroll
        for (int j = 0; j < TJ; ++j)
            sx[j] = static_cast<int>(*reinterpret_cast<const uint32_t *>(src + L::s + (BM + wn + 32 * j + r) * L::srow + 4 * g) & mask);
        const uint8_t *wl = src + wm * L::wrow, *xl = src + L::x + wn * L::xrow;
        mx_tile_step<0, XF, TI, TJ>(wl, xl, sw, sx, acc, r, g);
        mx_tile_step<1, XF, TI, TJ>(wl, xl, sw, sx, acc, r, g);
        mx_tile_step<2, XF, TI, TJ>(wl, xl, sw, sx, acc, r, g);
        mx_tile_step<3, XF, TI, TJ>(wl, xl, sw, sx, acc, r, g);
    };

    fill(0, lds);
    for (int t = 0; t < stages; ++t) {
        __syncthreads();         // stage t has come, and nobody reads the other buffer any more
        if (t + 1 < stages) fill(t + 1, lds + ((t + 1) & 1) * L::stage);
        multiply(t, lds + (t & 1) * L::stage);
    }

    // D: column r is a row of x, element v the weight row 8 (v / 4) + 4 g + v % 4
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
        const int n = wn + 32 * j + r;
        if (n >= rows) continue;
        T *row = static_cast<T *>(p.y) + (r0 + n) * p.M + m0;
#pragma unroll
        for (int i = 0; i < TI; i += WI) {
#pragma unroll
            for (int v = 0; v < 16; v += 4) {
                const int m = (wm + 32 * i) / WI + 2 * v + 4 * g;
                float out[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) out[q] = SILU ? silu_mul(acc[i][j][v + q], acc[i + WI - 1][j][v + q]) : acc[i][j][v + q];
                if (m < outs) put4(row + m, out, outs - m, p.vec);
            }
        }
    }
}

}  // namespace qg
