// mx_tile.hpp -- MX products for many rows: tiles of weights and activations
// brought from memory straight into LDS.
//
// A workgroup of WM x WN waves takes tiles of BM weight rows and BN rows of x in
// turn; a stage is 256 inputs of both in one of two LDS slots, filled by loads
// that go to LDS directly while others are multiplied. A wave takes BM / WM x BN
// / WN of the tile in blocks of 32 x 32. Stages run on from tile to tile: while
// a tile's results are written the next one's first stages are on their way.
//
// Which inputs an instruction takes together is free as long as both operands
// agree: of a stage's 8 blocks a lane with g = 0 takes blocks 0..3 in turn, one
// with g = 1 blocks 4..7. So its scales of the stage are the four bytes of one
// dword, and the instruction's byte selector walks them. Scales are laid out stage
// by stage first (mx_scales_kernel): of a row's line of scales a stage needs 8
// bytes, and a load costs by the lines it touches (fetched from the rows as they
// are, scales cost half as much as all codes).
//
// With SILU the tile's weight rows are 32 of the gate and 32 of the up matrix
// in turn, so that a lane holds both numbers of an output.
//
// Measured: 10240 x 17408 x 5120 e2m1 480 us (3.8 PFLOP/s; the instruction alone reaches
// 6.7), with SILU twice as many outputs 923; e4m3, two products each, 1265 (1.44, so
// 2.9 of 4.1). Of the 480 us the loads alone take 320, the products and LDS reads alone 370
// and the stores 60, which nothing overlaps: they leave the registers as they are
// issued, but the wait in the next tile's first stage is one for all memory
// operations. Experts of e2m1 rows, 64, 8 each, 2048 -> 2 x 1024: 96 us where 4096
// rows fill every tile, 107 where 4099 leave a nearly empty one each, 123 unevenly liked; e4m3
// 212, 229 and 243. Each stage is one block of instructions: with a branch in it the
// compiler moves the products of all four steps behind it, and the matrix cores wait
// while addresses are made (512 us). 256 x 128 tiles in three slots: 1024 x 2048 x 32768
// with SILU 91 us instead of 79; 128 x 128, two workgroups a compute unit, 94.
#pragma once

#include "mx_gemm.hpp"

namespace qg {

constexpr int kTileK = 256;      // inputs of a stage
constexpr int kTileScale = kTileK / kMxBlock;      // bytes of scales of a row and stage

constexpr int kTileSlots = 2;

template <int XF, bool GROUPED, int BM, int BN, int NW>
struct MxTileLds {
    static constexpr int wrow = kTileK / 2, xrow = static_cast<int>(mx_bytes<XF>(kTileK));
    static constexpr int wb = (BM + 127) / 128, xb = (BN + 127) / 128;    // loads of scales: 128 rows, 1 KiB
    static constexpr int x = BM * wrow, sw = x + BN * xrow, sx = sw + wb * 1024, stage = sx + xb * 1024;
    static constexpr int table = kTileSlots * stage, tables = GROUPED ? NW * 256 : 0;      // where rows of x begin, of two tiles
    static constexpr int bytes = table + 2 * tables + (GROUPED ? 256 : 0);        // (the last for what nobody wants)
};

// 16-byte chunk c of LDS row r lies at chunk c ^ swizzle(r): 16 lanes that
// read one chunk of 16 rows, or 8 of 8, meet no bank twice.
template <int CHUNKS>
__device__ __forceinline__ int mx_swizzle(int r)
{
    if constexpr (CHUNKS == 16) return r & 15;
    if constexpr (CHUNKS == 8) return (r & 7) ^ ((r >> 3) & 1);
    return (((r >> 1) ^ (r >> 2)) & 1) | ((((r >> 2) ^ (r >> 3)) & 1) << 1);
}

// The operands of one step (64 inputs) of a wave, from LDS (wl and xl: its first rows).
template <int XF, int TI, int TJ>
struct MxTileOps {
    static constexpr int XP = kXParts<XF>;
    u32x4 a[TI], b[TJ][XP];

    __device__ __forceinline__ void read(const uint8_t *wl, const uint8_t *xl, int s, int r, int g)
    {
        constexpr int wrow = kTileK / 2, xrow = static_cast<int>(mx_bytes<XF>(kTileK));
        // (the swizzle goes by a row's low four bits, which r has)
#pragma unroll
        for (int i = 0; i < TI; ++i)
            a[i] = *reinterpret_cast<const u32x4 *>(wl + (32 * i + r) * wrow + 16 * ((4 * g + s) ^ mx_swizzle<8>(r)));
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const uint8_t *row = xl + (32 * j + r) * xrow;
            if constexpr (XF == kMxE2M1) {
                b[j][0] = *reinterpret_cast<const u32x4 *>(row + 16 * ((4 * g + s) ^ mx_swizzle<8>(r)));
            } else {
                // bytes 0..15: half g of block s; bytes 16..31: half g of block 4 + s
                b[j][0] = *reinterpret_cast<const u32x4 *>(row + 16 * ((2 * s + g) ^ mx_swizzle<16>(r)));
                b[j][1] = *reinterpret_cast<const u32x4 *>(row + 16 * ((8 + 2 * s + g) ^ mx_swizzle<16>(r)));
            }
        }
    }
};

template <int S, int XF, int TI, int TJ>
__device__ __forceinline__ void mx_tile_step(const MxTileOps<XF, TI, TJ> &o, const int (&sw)[TI], const int (&sx)[TJ],
                                             f32x16 (&acc)[TI][TJ])
{
    constexpr int XP = kXParts<XF>;
    i32x8 b[TJ][XP];
#pragma unroll
    for (int j = 0; j < TJ; ++j) x_operands<XF>(o.b[j][0], o.b[j][XP - 1], b[j]);
#pragma unroll
    for (int h = 0; h < XP; ++h)
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            const i32x8 a = {int(o.a[i][0]), int(o.a[i][1]), int(o.a[i][2]), int(o.a[i][3]), 0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < TJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b[j][h], acc[i][j], kMxE2M1, XF, S, sw[i], S, sx[j]);
        }
}

// The instructions since the last of these in the order wanted: LDS reads (and
// LOADS loads to LDS) spread between the matrix instructions. Left alone the
// compiler puts every read right before its use, and the matrix cores wait.
template <int MFMAS, int READS, int LOADS>
__device__ __forceinline__ void mx_interleave()
{
    constexpr int slots = MFMAS < READS ? MFMAS : READS;
#pragma unroll
    for (int i = 0; i < slots; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, READS / slots, 0);                      // LDS reads
        if (LOADS / slots) __builtin_amdgcn_sched_group_barrier(0x020, LOADS / slots, 0);   // loads
        __builtin_amdgcn_sched_group_barrier(0x008, MFMAS / slots, 0);                      // matrix instructions
    }
    __builtin_amdgcn_sched_barrier(0);
}

// This wave's LDS reads are done, all but the last N of its memory operations too;
// then all waves of the workgroup meet. (One block, so that nothing moves between.)
template <int N>
__device__ __forceinline__ void mx_meet()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// A wave's part of a tile to memory: rows from n0 on of the tile's, outputs from
// m0 on. D: column r is a row of x, element v the weight row 8 (v / 4) + 4 g + v % 4; of
// bf16 two lanes of a row trade half of theirs, so that each stores 16 bytes side
// by side. Without branches (what lies outside goes to offsets out of range): cut
// into blocks, the compiler moves the accumulators about before it stores them.
// LINES: rows of y are whole pieces of 16 bytes.
template <typename T, bool SILU, bool LINES, int TI, int TJ>
__device__ __forceinline__ void mx_tile_store(const f32x16 (&acc)[TI][TJ], T *y, int64_t M, int rows, int outs, int n0, int m0)
{
    constexpr int WI = SILU ? 2 : 1, SIZE = static_cast<int>(sizeof(T));
    const int lane = mx_here(threadIdx.x & 63), r = lane & 31, g = lane >> 5;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
        const auto buf = mx_buffer(y + (n0 + 32 * j) * M, 32 * M * SIZE);
        const uint32_t row = n0 + 32 * j + r < rows ? static_cast<uint32_t>(r * M * SIZE) : kMxOut;
#pragma unroll
        for (int i = 0; i < TI; i += WI) {
            const int mb = m0 + 32 * i / WI;
            __builtin_amdgcn_sched_barrier(0);
            float out[16];
#pragma unroll
            for (int v = 0; v < 16; ++v) out[v] = !SILU ? acc[i][j][v] : SIZE == 4 ? silu_mul(acc[i][j][v], acc[i + WI - 1][j][v]) : silu_mul_bf16(acc[i][j][v], acc[i + WI - 1][j][v]);
            if constexpr (SIZE == 4) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int m = mb + 8 * q + 4 * g;
                    if constexpr (LINES) {
                        const f32x4 v = {out[4 * q], out[4 * q + 1], out[4 * q + 2], out[4 * q + 3]};
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), buf, m < outs ? row + m * 4 : kMxOut, 0, 0);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(out[4 * q + e]), buf, m + e < outs ? row + (m + e) * 4 : kMxOut, 0, 0);
                    }
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    // this lane's outputs 8 q + 4 g .. and 8 (q + 1) + 4 g ..
                    u32x2 lo, hi;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const auto t = __builtin_amdgcn_permlane32_swap(f32_to_bf16_pair(out[4 * q + 2 * e], out[4 * q + 2 * e + 1]),
                                                                        f32_to_bf16_pair(out[4 * q + 4 + 2 * e], out[4 * q + 5 + 2 * e]), false, false);
                        lo[e] = t[0], hi[e] = t[1];
                    }
                    // now 8 (q + g) .. + 7
                    const int m = mb + 8 * (q + g);
                    const u32x4 v = {lo[0], lo[1], hi[0], hi[1]};
                    if constexpr (LINES) {
                        __builtin_amdgcn_raw_buffer_store_b128(v, buf, m < outs ? row + m * 2 : kMxOut, 0, 0);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(v[e / 2] >> (16 * (e & 1))), buf,
                                                                  m + e < outs ? row + (m + e) * 2 : kMxOut, 0, 0);
                    }
                }
            }
        }
    }
}

// A tile: rows r0 .. r0 + rows - 1 of expert e, outputs from m0 on.
struct MxTile {
    int r0, m0, e, rows;      // rows 0: none
};

// Scales of rows as the tiles take them: [stage][row][8], zeros behind a row's
// end. Weights' rows, then x's, which with `order` are those of the sorted pairs.
struct MxScalesParams {
    const uint8_t *ws, *xs;
    uint8_t *to_w, *to_x;
    int64_t wrows, xrows;     // x: rows of the product
    int32_t wblocks;          // workgroups that take weights' rows
    int32_t pitch, blocks;    // bytes of a row, of these scales
    int32_t stages;
    const int32_t *order;
    int64_t x_rows;           // rows that may be gathered
    uint32_t *x_at;           // with `order`: where each row's codes begin, or kMxOut
    int32_t xrb;              // bytes of a row's codes
    FastDiv top;
    // grouped: the list of tiles of BN rows
    int32_t xblocks;          // workgroups that take x's rows; those behind list tiles
    const int32_t *offsets;
    int32_t experts, tiles_n, bn;
    MxTileEntry *tiles;
};

// A tile of rows: rows r0 .. r0 + rows - 1 of expert e; rows 0: none.
struct MxTileEntry {
    int32_t e, r0, rows, pad;
};

constexpr int kScaleThreads = 256;

__device__ __forceinline__ void mx_scales_rows(const MxScalesParams &p, const uint8_t *from, uint8_t *to, int64_t rows, int64_t first, bool gather)
{
    // lanes along rows, so that stores lie side by side; of a row 16 bytes, two stages', at once
    const int64_t row = first + (threadIdx.x & 63);
    if (row >= rows) return;
    int64_t at = threadIdx.x & 63;
    if (gather) {
        const int64_t pair = p.order[row];
        at = pair < 0 || pair >= rows ? -1 : static_cast<uint32_t>(pair) / p.top;
        if (at >= p.x_rows) at = -1;
        if (threadIdx.x < 64) p.x_at[row] = at < 0 ? kMxOut : static_cast<uint32_t>(at * p.xrb);
    }
    const auto buf = mx_buffer(from + (gather ? 0 : first * p.pitch), (gather ? p.x_rows : min(int64_t(64), rows - first)) * p.pitch);
    for (int t = threadIdx.x >> 6; 2 * t < p.stages; t += kScaleThreads / 64) {
        u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, at < 0 ? kMxOut : static_cast<uint32_t>(at * p.pitch + 16 * t), 0, 0));
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int left = p.blocks - (16 * t + 4 * d);
            if (left < 4) v[d] &= left <= 0 ? 0 : (1u << (8 * left)) - 1;
        }
        *reinterpret_cast<u32x2 *>(to + (2 * t * rows + row) * 8) = u32x2{v[0], v[1]};
        if (2 * t + 1 < p.stages) *reinterpret_cast<u32x2 *>(to + ((2 * t + 1) * rows + row) * 8) = u32x2{v[2], v[3]};
    }
}

// Every expert's rows in tiles, expert by expert: a thread finds one tile's expert
// in the running sums of tiles (offsets out of range are cut, so that any
// contents give rows in [0, pairs)).
__device__ __forceinline__ void mx_list_tiles(const MxScalesParams &p, int first)
{
    __shared__ int upto[kMaxExperts];                // tiles of the experts up to each
    __shared__ int waves[kScaleThreads / 64];
    constexpr int C = kMaxExperts / kScaleThreads;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, most = static_cast<int>(p.xrows);
    const auto place = [&](int e) { return max(0, min(p.offsets[min(e, p.experts)], most)); };
    int o[C + 1], mine = 0;
#pragma unroll
    for (int j = 0; j <= C; ++j) o[j] = place(threadIdx.x * C + j);
#pragma unroll
    for (int j = 0; j < C; ++j) mine += (max(o[j + 1] - o[j], 0) + p.bn - 1) / p.bn;
    int sum = wave_inclusive_sum32(mine);
    if (lane == 63) waves[wave] = sum;
    __syncthreads();
    for (int w = 0; w < wave; ++w) sum += waves[w];
    sum -= mine;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        sum += (max(o[j + 1] - o[j], 0) + p.bn - 1) / p.bn;
        upto[threadIdx.x * C + j] = sum;
    }
    __syncthreads();
    const int tile = first + threadIdx.x;
    // behind the list the number of tiles that there are
    if (tile == 0) p.tiles[p.tiles_n] = MxTileEntry{max(0, min(upto[kMaxExperts - 1], p.tiles_n)), 0, 0, 0};
    if (tile >= p.tiles_n) return;
    int lo = 0, hi = kMaxExperts;                    // the first expert with more tiles up to it
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (upto[mid] > tile) hi = mid;
        else lo = mid + 1;
    }
    MxTileEntry t{0, 0, 0, 0};
    if (lo < p.experts) {
        const int begin = place(lo), rows = max(place(lo + 1) - begin, 0), nth = tile - (lo ? upto[lo - 1] : 0);
        // (no plan's offsets may make the sums run over)
        if (nth >= 0 && nth < (rows + p.bn - 1) / p.bn) {
            t.e = lo;
            t.r0 = begin + nth * p.bn;
            t.rows = min(p.bn, rows - nth * p.bn);
        }
    }
    p.tiles[tile] = t;
}

static __global__ __launch_bounds__(kScaleThreads) void mx_scales_kernel(MxScalesParams p)
{
    const int block = blockIdx.x;
    if (block < p.wblocks)
        mx_scales_rows(p, p.ws, p.to_w, p.wrows, int64_t(block) * 64, false);
    else if (block < p.wblocks + p.xblocks)
        mx_scales_rows(p, p.xs, p.to_x, p.xrows, int64_t(block - p.wblocks) * 64, p.order != nullptr);
    else
        mx_list_tiles(p, (block - p.wblocks - p.xblocks) * kScaleThreads);
}

template <int XF, typename T, bool SILU, bool GROUPED, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM *WN) void mx_tile_kernel(MxGemmParams p)
{
    constexpr int NW = WM * WN, TI = BM / WM / 32, TJ = BN / WN / 32, WI = SILU ? 2 : 1, D = kTileSlots;
    using L = MxTileLds<XF, GROUPED, BM, BN, NW>;
    static_assert(TI % WI == 0, "a wave holds gate and up rows of an output");
    constexpr int OUTS = BM / WI;                    // outputs of a tile
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, g = lane >> 5;
    const int wrb = p.K / 2, xrb = static_cast<int>(mx_bytes<XF>(p.K));
    const int stages = (p.K + kTileK - 1) / kTileK;
    const bool gather = GROUPED && p.order;

    // Consecutive workgroups go to the 8 XCDs in turn: each XCD gets a run of
    // tiles, which its workgroups take in turn, in bands of 4 tiles of rows, these
    // first: the 32 tiles that an XCD's compute units work on are 8 x 4, 12
    // operands for 33 in a row.
    int nth = blockIdx.x >> 3;
    // f(first id of the XCD's run, its end, workgroups of the XCD)
    const int tiles_n = GROUPED ? p.tiles[p.tiles_n].e : p.tiles_n;
    const auto run = [&](auto f) {
        const int ntiles = p.tiles_m * tiles_n, xcd = blockIdx.x & 7, xcds = min(8, static_cast<int>(gridDim.x));
        f(xcd * (ntiles / xcds) + min(xcd, ntiles % xcds), ntiles / xcds + (xcd < ntiles % xcds), (static_cast<int>(gridDim.x) - xcd + 7) >> 3);
    };
    constexpr int BAND = 4;
    const auto place = [&](int id, int &tm, int &tn) {
        const int band = id / (BAND * p.tiles_m), in = id - band * (BAND * p.tiles_m);
        const int high = min(BAND, tiles_n - band * BAND);
        tm = in / high, tn = band * BAND + in % high;
    };
    // grouped: the workgroup's next 64 tiles, one a lane, and those not taken yet, so that
    // a new tile asks for nothing in memory while others' loads are under way (these
    // come in order: the wait for one is a wait for all before it)
    MxTile mine{0, 0, 0, 0};
    uint64_t untaken = 0;
    const auto next_tile = [&]() __attribute__((always_inline)) {
        MxTile t{0, 0, 0, 0};
        if constexpr (GROUPED) {
            if (untaken == 0)
                run([&](int first, int n, int step) {
                    const int lane = mx_here(threadIdx.x & 63);
                    while (untaken == 0 && nth < n) {
                        int tm, tn;
                        place(first + min(nth + lane * step, n - 1), tm, tn);
                        const MxTileEntry u = p.tiles[tn];
                        mine = MxTile{u.r0, tm * OUTS, u.e, u.rows};
                        untaken = __ballot(nth + lane * step < n && u.rows > 0);
                        nth += 64 * step;
                    }
                });
            if (untaken != 0) {
                const int from = __builtin_ctzll(untaken);
                untaken &= untaken - 1;
                t.r0 = __builtin_amdgcn_readlane(mine.r0, from);
                t.m0 = __builtin_amdgcn_readlane(mine.m0, from);
                t.e = __builtin_amdgcn_readlane(mine.e, from);
                t.rows = __builtin_amdgcn_readlane(mine.rows, from);
            }
        } else {
            run([&](int first, int n, int step) {
                if (nth >= n) return;
                int tm, tn;
                place(first + nth, tm, tn);
                nth += step;
                t.m0 = tm * OUTS;
                t.r0 = tn * BN;
                t.rows = static_cast<int>(min(int64_t(BN), p.N - t.r0));
            });
        }
        return t;
    };

    // This lane's pieces of a stage. Weights: load i of the wave fills 8 LDS rows
    // from 8 q on, q = i * NW + wave; x likewise; scales 128 rows, two a lane.
    constexpr int WL = BM / 8 / NW, XR = 1024 / L::xrow, XL = BN / XR / NW, XC = L::xrow / 16;
    constexpr int SB = L::wb + L::xb;
    static_assert(SB <= NW, "a load of scales a wave");
    const int sload = wave % SB;                     // (two waves may have the same)
    const bool sofw = sload < L::wb;
    static_assert(WL * NW * 8 == BM && XL * NW * XR == BN, "whole loads");
    const auto weight_row = [&](int row) { return SILU ? (row >> 6) * 32 + (row & 31) : row; };
    // the row of x's load i that this lane fills, and the piece of it
    const auto x_lds_row = [&](int lane, int i) { return XR * (i * NW + wave) + lane / XC; };
    const auto x_piece = [&](int lane, int i) { return (lane % XC) ^ mx_swizzle<XC>(x_lds_row(lane, i)); };
    // the tile that is being loaded, and its next stage
    int at = 0;
    const uint8_t *wbase[WI], *xbase;
    int wlen, xlen;
    // this wave's load of scales: rows behind `sbase` of those laid out
    const uint8_t *sbase;
    int64_t srows;           // rows of a stage
    int slen;
    // Gathered rows: of a tile's rows that this wave loads, one a lane, where they begin,
    // in one of two tables in LDS, asked for one fill before the first that takes it.
    int turn = 1;            // the table of the tile that is being loaded
    static_assert(BN / NW <= 64, "a lane a row");
    const auto ask = [&](const MxTile &t, int table, bool wanted) __attribute__((always_inline)) {
        const int lane = mx_here(threadIdx.x & 63);
        // (what lies out of range comes as zeros)
        mx_to_lds4(mx_buffer(p.x_at + t.r0, wanted && gather ? t.rows * 4 : 0), lds + L::table + (wanted ? table * L::tables + wave * 256 : 2 * L::tables),
                   mx_in_or_out(4 * (XR * (lane / XR * NW + wave) + lane % XR), lane, BN / NW));
    };
    const auto open = [&](const MxTile &t) {
        at = 0;
        turn ^= 1;
        const int outs = min(OUTS, static_cast<int>(p.M) - t.m0);
#pragma unroll
        for (int i = 0; i < WI; ++i) wbase[i] = p.wc + ((int64_t(t.e) * WI + i) * p.M + t.m0) * wrb;
        wlen = outs * wrb;
        const int64_t first = gather ? 0 : t.r0, in = gather ? p.x_rows : t.rows;
        xbase = p.xc + first * xrb;
        xlen = static_cast<int>(in * xrb);
        // (of the weights' scales the up matrix's come after all of the gate's)
        const int64_t srow = sofw ? int64_t(t.e) * WI * p.M + t.m0 + 128 / WI * sload : t.r0 + 128 * (sload - L::wb);
        sbase = (sofw ? p.ws : p.xs) + srow * kTileScale;
        srows = sofw ? p.ws_rows : p.N;
        slen = static_cast<int>(max(min(srows - srow, sofw ? (WI - 1) * p.M + OUTS : int64_t(BN)), int64_t(0)) * kTileScale);
    };
    MxTile after;            // to be opened next
    // a lane's scales are of two rows of the weights' LDS rows, or of x's
    const int silu_soff = SILU ? mx_here(static_cast<int>((sofw ? weight_row(2 * lane) + (lane & 16 ? p.M : 0) : 2 * lane) * kTileScale)) : 0;
    const uint32_t gathers = GROUPED ? mx_here(gather ? -1 : 0) : 0;
    // (without branches: a stage is one block of instructions, of which the matrix
    // instructions are spread over all the others)
    const auto fill = [&](uint8_t *dst, bool real) __attribute__((always_inline)) {
        const int wk = at * L::wrow, xk0 = at * L::xrow;
        const int wrb = mx_here_scalar(p.K / 2), xrb = static_cast<int>(mx_bytes<XF>(mx_here_scalar(p.K)));
        const int left = p.K - at * kTileK, lane = mx_here(threadIdx.x & 63);
        __amdgpu_buffer_rsrc_t wbuf[WI];
#pragma unroll
        for (int i = 0; i < WI; ++i) wbuf[i] = mx_buffer(wbase[i] + wk, real ? wlen - wk : 0);
        const auto xbuf = mx_buffer(xbase + xk0, real ? xlen - xk0 : 0);
        // Within a load rows lie side by side, so that a lane has one offset for all of
        // the weights' (the swizzle goes by a row's low four bits, and NW is even).
        const uint32_t woff = static_cast<uint32_t>((lane >> 3) * wrb + 16 * ((lane & 7) ^ mx_swizzle<8>(8 * wave + (lane >> 3))));
#pragma unroll
        for (int i = 0; i < WL; ++i) {
            const int q = i * NW + wave, part = SILU ? (q >> 2) & 1 : 0;
            mx_to_lds16(wbuf[part], dst + q * 1024, woff + weight_row(8 * q) * wrb);
        }
        // inputs behind the row's end are zeros (the weights' there are any finite numbers)
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int q = i * NW + wave, piece = x_piece(lane, i);
            uint32_t row = static_cast<uint32_t>(lane / XC * xrb + XR * q * xrb);
            if constexpr (GROUPED) {
                const uint32_t *table = reinterpret_cast<const uint32_t *>(lds + L::table + turn * L::tables + wave * 256);
                const uint32_t from = table[XR * i + lane / XC];
                row = (from & gathers) | (row & ~gathers);
            }
            mx_to_lds16(xbuf, dst + L::x + q * 1024, mx_in_or_out(row + 16 * piece, piece * (XF == kMxE2M1 ? 32 : 16), left));
        }
        mx_to_lds16(mx_buffer(sbase + at * srows * kTileScale, real ? slen : 0), dst + L::sw + sload * 1024,
                    SILU ? silu_soff : 2 * kTileScale * lane);
        if constexpr (GROUPED) ask(after, turn ^ 1, at + 1 == stages);
    };

    f32x16 acc[TI][TJ];
    // (waves of the same rows next to each other, so that where a tile has half of its
    // rows every SIMD is left one of its waves)
    const int wm = (wave % WM) * (BM / WM), wn = (wave / WM) * (BN / WN);
    int sw[2][TI], sx[2][TJ];
    MxTileOps<XF, TI, TJ> ops[2];
    // step 0 of the stage in a slot and the stage's scales
    const auto begin = [&](int slot, int (&w)[TI], int (&x)[TJ]) {
        const uint8_t *src = lds + slot * L::stage, *swsrc = src + L::sw + 4 * g, *sxsrc = src + L::sx + 4 * g;
#pragma unroll
        for (int i = 0; i < TI; ++i) w[i] = *reinterpret_cast<const int *>(swsrc + (wm + 32 * i + r) * kTileScale);
#pragma unroll
        for (int j = 0; j < TJ; ++j) x[j] = *reinterpret_cast<const int *>(sxsrc + (wn + 32 * j + r) * kTileScale);
        ops[0].read(src + wm * L::wrow, src + L::x + wn * L::xrow, 0, r, g);
    };

    // tiles that are loaded, at least in part, behind the current one
    MxTile cur = next_tile(), ahead[D];
    if (cur.rows == 0) return;
    int waiting = 0;
    bool more = true;
    after = next_tile();
    if constexpr (GROUPED) {
        ask(cur, 0, true);
        ask(after, 1, true);
        mx_meet<0>();
    }
    open(cur);
    // takes the next stage's tile
    const auto advance = [&]() __attribute__((always_inline)) {
        if (!more || at < stages) return;
        more = after.rows != 0;
        if (!more) return;
        open(after);
#pragma unroll
        for (int i = 0; i < D; ++i)
            if (i == waiting) ahead[i] = after;
        ++waiting;
        after = next_tile();
    };
    for (int d = 0; d < D; ++d) {
        advance();
        fill(lds + d * L::stage, more);
        at += more;
    }
    mx_meet<0>();
    begin(0, sw[0], sx[0]);

    // A step's operands are read while the one before is multiplied. Once the
    // last step's are read the waves meet: then the next stage's first operands
    // are read and the stage's slot is filled anew, beside the last step's products.
    constexpr int MFMAS = TI * TJ * kXParts<XF>, READS = TI + TJ * kXParts<XF>, LOADS = WL + XL + 1 + GROUPED;
    int slot = 0;
    const auto stage = [&]() __attribute__((always_inline)) {
        const uint8_t *wl = lds + slot * L::stage + wm * L::wrow, *xl = lds + slot * L::stage + L::x + wn * L::xrow;
        advance();
        __builtin_amdgcn_sched_barrier(0);
        ops[1].read(wl, xl, 1, r, g);
        mx_tile_step<0>(ops[0], sw[0], sx[0], acc);
        mx_interleave<MFMAS, READS, 0>();
        ops[0].read(wl, xl, 2, r, g);
        mx_tile_step<1>(ops[1], sw[0], sx[0], acc);
        mx_interleave<MFMAS, READS, 0>();
        ops[1].read(wl, xl, 3, r, g);
        mx_tile_step<2>(ops[0], sw[0], sx[0], acc);
        mx_interleave<MFMAS, READS, 0>();
        mx_meet<0>();
        __builtin_amdgcn_sched_barrier(0);
        const int freed = slot;
        slot = slot + 1 == D ? 0 : slot + 1;
        begin(slot, sw[1], sx[1]);
        fill(lds + freed * L::stage, more);
        mx_tile_step<3>(ops[1], sw[0], sx[0], acc);
        mx_interleave<MFMAS, READS + TI + TJ, LOADS>();
        at += more;
#pragma unroll
        for (int i = 0; i < TI; ++i) sw[0][i] = sw[1][i];
#pragma unroll
        for (int j = 0; j < TJ; ++j) sx[0][j] = sx[1][j];
    };
    // a wave that has no rows of the tile brings its share of the loads
    const auto idle_stage = [&]() __attribute__((always_inline)) {
        advance();
        mx_meet<0>();
        const int freed = slot;
        slot = slot + 1 == D ? 0 : slot + 1;
        begin(slot, sw[0], sx[0]);
        fill(lds + freed * L::stage, more);
        at += more;
    };
    for (;;) {
        if (wn < cur.rows) {
#pragma unroll
            for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int j = 0; j < TJ; ++j)
#pragma unroll
                    for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
            for (int t = 0; t < stages; ++t) stage();
            const int outs = min(OUTS, static_cast<int>(p.M) - cur.m0);
            if (p.M % (16 / static_cast<int>(sizeof(T))) == 0)
                mx_tile_store<T, SILU, true>(acc, static_cast<T *>(p.y) + int64_t(cur.r0) * p.M + cur.m0, p.M, cur.rows, outs, wn, wm / WI);
            else
                mx_tile_store<T, SILU, false>(acc, static_cast<T *>(p.y) + int64_t(cur.r0) * p.M + cur.m0, p.M, cur.rows, outs, wn, wm / WI);
        } else {
            for (int t = 0; t < stages; ++t) idle_stage();
        }
        if (waiting == 0) break;
        cur = ahead[0];
#pragma unroll
        for (int i = 0; i + 1 < D; ++i) ahead[i] = ahead[i + 1];
        --waiting;
    }
}

}  // namespace qg
