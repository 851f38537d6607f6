// attn_rows.hpp -- attention for many query rows of a request and key/value
// head: chunks of a prompt.
//
// The four waves of a workgroup have 16 QT rows each and go over the same
// tiles of tokens. What bounds it is the vector unit (of a row and token:
// 18 to 19 instructions a lane at 128 channels in float32, where the matrix
// products take 512 flop twice): so the codes are made operands once for the
// four waves, a quarter by each, and left in LDS in operand order, and every
// wave then reads its operands by 16-byte reads of consecutive lanes. K's
// codes are fetched in operand order already (a lane takes 8 bytes of the
// token its row is); V's go through a wave's own piece of LDS to be
// transposed. Tiles are double buffered: one barrier a tile.
//
// 2048 float32 rows after 8192 tokens, 32 heads of 128 channels: 737 us (618
// GFLOP in two pieces, 0.84 PFLOP/s; vector unit 58% and matrix cores 33% busy,
// seldom both). Six bfloat16 prompts of up to 4001 tokens, 32 heads of 64
// channels: 514 us (vector unit 76%: a quarter-rate exponential and 8.5 other
// instructions a score; matrix cores 20%).
#pragma once

#include "attn_common.hpp"

namespace qg {

// Tokens of a tile: the operands of a tile are 16 or 32 KiB.
constexpr int rows_tile_tokens(int dim) { return dim == 256 ? 32 : 64; }

template <int D>
struct RowsTile {
    static constexpr int kTok = rows_tile_tokens(D), NG = D / 64;
    u32x4 k[kTok / 16][NG][2][64];                         // [block of 16 tokens][group][half of its channels][lane]
    u32x4 v[kTok / 32][D / 16][64];                        // [block of 32 tokens][block of 16 channels][lane]
};

// Coefficients of a tile: they are put into LDS a tile ahead of the codes, so
// that the choice of the loop for a tile comes before its codes are waited for.
template <int D>
struct RowsCoefs {
    static constexpr int kTok = rows_tile_tokens(D), NG = D / 64;
    alignas(16) float co[2][NG][2][kTok];                  // as in attn_few.hpp
    int32_t out[kTok / 32];                                // the last of its tiles with value scales out of the range, by halves
};

template <int D>
struct RowsLds {
    static constexpr int kRaw = 32 * (D == 64 ? 16 : 32);   // code bytes of V a wave transposes
    RowsTile<D> tile[2];
    RowsCoefs<D> coefs[3];
    uint8_t raw[4][kRaw];
    TileSizes sizes[4];                                    // a wave's notes of a careful step, and its rows' tokens
    int32_t pos[4][32];
};

template <typename T, int D, int QT>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_rows_kernel(AttnParams p)
{
    constexpr bool kTwo = sizeof(T) == 4;
    constexpr int kTok = rows_tile_tokens(D), NG = D / 64, NB = kTok / 16, NH = kTok / 32;
    constexpr int R = 64 * QT;
    constexpr int kRow = D / 2;
    constexpr int KG = D == 256 ? 2 : NG;                   // groups of K a wave makes operands of
    constexpr int VB = D == 64 ? 16 : 32;                   // bytes of a token's V codes a wave transposes
    extern __shared__ __align__(16) uint8_t lds_bytes[];
    RowsLds<D> &lds = *reinterpret_cast<RowsLds<D> *>(lds_bytes);

    int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kv_head = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.kv.heads));
    RowTile t;
    if (!find_tile<R>(p, blockIdx.x / static_cast<unsigned>(p.kv.heads), t)) return;
    int32_t begin, end;
    if (!split_tokens(p, t, kTok, begin, end)) return;
    const int tiles = (end - begin + kTok - 1) / kTok;

    QueryRows<T, D, QT> rows;
    const uint32_t first_row = t.row0 + wave * 16 * QT;
    TileSizes &sizes = lds.sizes[wave];
    int32_t *const pos = lds.pos[wave];
    rows.load(p, t, kv_head, first_row, lane, pos);

    // ---- fetching: K block `wave` (mod NB) of the tile, V's codes of 32 tokens
    // and a part of the channels, coefficients of the K block's tokens
    const int32_t *row_pages = p.table + int64_t(t.b) * p.table_stride;
    const uint8_t *const data = p.kv.data + int64_t(kv_head) * p.kv.block_bytes;
    const int32_t half = p.kv.block_bytes >> 1;
    const int page_mask = (1 << p.kv.page_shift) - 1;
    const int k_block = wave % NB, k_group = D == 256 ? wave / NB * KG : 0;
    const int v_half = NH == 2 ? wave >> 1 : 0, v_part = NH == 2 ? wave & 1 : wave;
    // lane j: the page of block j (mod NB) of a tile
    auto fetch_pages = [&](int tile) {
        const int32_t want = begin + tile * kTok + (lane & (NB - 1)) * 16;
        return row_pages[(want < end ? want : end - 1) >> p.kv.page_shift];
    };
    int32_t next_pages = 0, far_pages = 0;                  // of the next tile and of the one behind it
    u32x2 k_raw[KG];
    uint32_t v_raw[2][VB / 16];
    uint32_t coef[NG];
    bool coef_known = true;
    auto block = [&](int32_t base, int32_t pages, int blk, bool &known, int &at) {
        const int32_t id = __builtin_amdgcn_readlane(pages, blk);
        known = static_cast<uint32_t>(id) < static_cast<uint32_t>(p.kv.num_pages);
        at = (base + blk * 16) & page_mask;
        return data + (known ? id : 0) * p.kv.page_bytes;
    };
    auto fetch_codes = [&](int tile, int32_t pages) __attribute__((always_inline)) {
        const int32_t base = begin + tile * kTok;
        bool known;
        int at;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint8_t *src = block(base, pages, v_half * 2 + j, known, at) + half + at * kRow + v_part * VB +
                                 static_cast<uint32_t>((lane >> 2) * kRow + (lane & 3) * (VB / 4));
            if constexpr (VB == 32) {
                const u32x2 v = *reinterpret_cast<const u32x2 *>(src);
                v_raw[j][0] = v[0], v_raw[j][1] = v[1];
            } else {
                v_raw[j][0] = *reinterpret_cast<const uint32_t *>(src);
            }
        }
        const uint8_t *page = block(base, pages, k_block, known, at);
#pragma unroll
        for (int g = 0; g < KG; ++g)
            k_raw[g] = *reinterpret_cast<const u32x2 *>(page + at * kRow + (k_group + g) * 32 +
                                                        static_cast<uint32_t>((lane & 15) * kRow + (lane >> 4) * 8));
    };
    auto fetch_coefs = [&](int tile, int32_t pages) __attribute__((always_inline)) {
        if (NB == 4 || wave < NB) {
            int at;
            const uint8_t *page = block(begin + tile * kTok, pages, k_block, coef_known, at);
            load_coefs(page + ((D / 2) << p.kv.page_shift) + at * (D / 16) +
                           static_cast<uint32_t>(((lane >> 4) & 1) * half + (lane & 15) * (D / 16)),
                       coef);
        }
    };
    int E = kAbove;                                         // range of plain tiles' value scales, up to 4 at first
    auto put_coefs = [&](RowsCoefs<D> &s, int tile) __attribute__((always_inline)) {
        if (NB == 4 || wave < NB) {
            bool in = true;
            const bool inside = begin + tile * kTok + k_block * 16 + (lane & 15) < end;
            const bool is_v = (lane >> 4) & 1;
            const float odd = is_v && (lane & 1) ? 0.0625f : 1.0f, centre = is_v && (lane & 1) ? kOddCentre : 8.0f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint32_t co = coef_of(coef[g], coef_known, inside);
                const float sc = __uint_as_float(co << 16), bi = __uint_as_float(co & 0xffff0000u);
                in = in & in_range(co, E);
                if (lane < 32) {
                    s.co[is_v][g][0][k_block * 16 + (lane & 15)] = sc * odd;
                    s.co[is_v][g][1][k_block * 16 + (lane & 15)] = kTwo ? fmaf(centre, sc, bi) : bi;
                }
            }
            if ((__ballot(in) >> 16 & 0xffff) != 0xffff) s.out[k_block / 2] = tile;      // the lanes of V
        }
    };
    const NibbleBits bits;
    auto put_tile = [&](RowsTile<D> &s) __attribute__((always_inline)) {
        uint8_t *raw = lds.raw[wave];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint8_t *dst = raw + (j * 16 + (lane >> 2)) * VB + (lane & 3) * (VB / 4);
            if constexpr (VB == 32) *reinterpret_cast<u32x2 *>(dst) = u32x2{v_raw[j][0], v_raw[j][1]};
            else *reinterpret_cast<uint32_t *>(dst) = v_raw[j][0];
        }
        wave_fence();
#pragma unroll
        for (int g = 0; g < KG; ++g)
#pragma unroll
            for (int st = 0; st < 2; ++st)
                s.k[k_block][k_group + g][st][lane] =
                    __builtin_bit_cast(u32x4, nibbles<kTwo>(st ? static_cast<uint32_t>(k_raw[g][1]) : static_cast<uint32_t>(k_raw[g][0]), bits));
        // lane: token 16 (i / 4 % 2) + 4 (lane / 16) + i % 4 of i = lane % 16,
        // the 8 bytes of two blocks of channels in turn
        const int i = lane & 15, tok = ((i >> 2) & 1) * 16 + (lane >> 4) * 4 + (i & 3);
#pragma unroll
        for (int n = 0; n < VB / 16; ++n) {
            const i32x2 w = read_transposed(raw + tok * VB + (n * 2 + (i >> 3)) * 8);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                s.v[v_half][v_part * (VB / 8) + n * 2 + h][lane] =
                    __builtin_bit_cast(u32x4, nibbles<kTwo, kOddCentre>(h ? static_cast<uint32_t>(w[1]) : static_cast<uint32_t>(w[0]), bits));
        }
        wave_fence();
    };

    // ---- 32 tokens: from block 2 hb of the tile on; QN tiles of rows from the first
    auto compute = [&](const RowsTile<D> &s, const RowsCoefs<D> &c, int hb, int32_t base, auto care_tag, int first, auto rows_tag) __attribute__((always_inline)) {
        constexpr bool kCareful = decltype(care_tag)::value;
        constexpr int QN = decltype(rows_tag)::value;
        const int g4 = lane >> 4;
        f32x4 x[QN][2];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const f16x8 k0 = __builtin_bit_cast(f16x8, s.k[hb * 2 + a][g][0][lane]);
                const f16x8 k1 = __builtin_bit_cast(f16x8, s.k[hb * 2 + a][g][1][lane]);
                const f32x4 sc = *reinterpret_cast<const f32x4 *>(&c.co[0][g][0][(hb * 2 + a) * 16 + g4 * 4]);
                const f32x4 bi = *reinterpret_cast<const f32x4 *>(&c.co[0][g][1][(hb * 2 + a) * 16 + g4 * 4]);
#pragma unroll
                for (int q = 0; q < QN; ++q) rows.score(first + q, g, k0, k1, sc, bi, x[q][a]);
            }
        uint32_t visible[QN] = {};
#pragma unroll
        for (int q = 0; q < QN; ++q)
            rows.template weigh<kCareful>(p, first + q, kCareful ? pos[(first + q) * 16 + (lane & 15)] : 0, x[q], visible[q],
                                          &sizes, 0, E, base, g4);
        // small groups of vector and matrix instructions in turn (2048 float32
        // rows after 8192 cached tokens: 736 us, 751 without; with one product a
        // piece, bfloat16, the compiler's own order is better, 513 and 549, and with
        // 256 channels, 45.9 and 47.6)
        if constexpr (kTwo && D < 256) __builtin_amdgcn_iglp_opt(0);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f16x8 ph[QN], pl[QN];
            f32x4 sc[2], bi[2];
            float down[QN];
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                sc[a] = *reinterpret_cast<const f32x4 *>(&c.co[1][g][0][(hb * 2 + a) * 16 + g4 * 4]);
                bi[a] = *reinterpret_cast<const f32x4 *>(&c.co[1][g][1][(hb * 2 + a) * 16 + g4 * 4]);
            }
#pragma unroll
            for (int q = 0; q < QN; ++q)
                rows.template pieces<kCareful>(first + q, g, x[q][0], x[q][1], visible[q], sc, bi, ph[q], pl[q], down[q]);
#pragma unroll
            for (int db = 0; db < 4; ++db) {
                const f16x8 v[1] = {__builtin_bit_cast(f16x8, s.v[hb][g * 4 + db][lane])};
#pragma unroll
                for (int q = 0; q < QN; ++q) rows.template add<kCareful>(first + q, g * 4 + db, v, &ph[q], &pl[q], down[q]);
            }
        }
    };

    if (tiles > 0) {
        const int32_t first_pages = fetch_pages(0);
        if (tiles > 1) next_pages = fetch_pages(1);
        fetch_coefs(0, first_pages);
        fetch_codes(0, first_pages);
        if (threadIdx.x < 3 * NH) lds.coefs[threadIdx.x / NH].out[threadIdx.x % NH] = -1;
        __syncthreads();
        put_coefs(lds.coefs[0], 0);
        if (tiles > 1) fetch_coefs(1, next_pages);
        if (tiles > 2) far_pages = fetch_pages(2);
        __syncthreads();
    }
    const int steps = (end - begin + 31) / 32;
    // Whether the value scales of the tile in LDS, and of the next one, are in the
    // range (bits: its halves; looked up when the coefficients are there, so that
    // no step waits). kStale: looked at with an earlier range, and careful.
    constexpr int kStale = 4;
    auto ranges = [&](const int32_t (&out)[NH], int tile) {
        int in = 0;
#pragma unroll
        for (int h = 0; h < NH; ++h) in |= __builtin_amdgcn_readfirstlane(out[h]) != tile ? 1 << h : 0;
        return in;
    };
    int in = 0, next_in = steps > 0 ? ranges(lds.coefs[0].out, 0) : 0;
    auto whole = [&](int32_t base, int count) { return base + count <= end && all_visible(p, t, base, count); };
    // whether a step needs no care: every row sees all of its tokens, and the
    // value scales are in the range
    auto plain = [&](int step) {
        const int now = in & 2, then = next_in & 1;
        return (step % NH == 0 ? then : now) != 0 && whole(begin + step * 32, 32);
    };
    auto advance = [&](int step, auto care_tag) __attribute__((always_inline)) {
        // the lane number is made opaque anew: offsets made from it are then
        // not kept in registers through the loop
        asm volatile("" : "+v"(lane));
        const int i = step / NH, hb = step % NH;
        RowsTile<D> &s = lds.tile[i & 1];
        if (hb == 0) {
            put_tile(s);
            if (i + 1 < tiles) put_coefs(lds.coefs[(i + 1) % 3], i + 1);
            __syncthreads();
            in = next_in;
            int32_t out[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h) out[h] = lds.coefs[(i + 1) % 3].out[h];
            if (i + 1 < tiles) {
                fetch_codes(i + 1, next_pages);
                next_pages = far_pages;
                if (i + 2 < tiles) fetch_coefs(i + 2, next_pages);
                if (i + 3 < tiles) far_pages = fetch_pages(i + 3);
            }
            next_in = ranges(out, i + 1);
        }
        if constexpr (decltype(care_tag)::value) {
            const float size = note_sizes<NG>(sizes, &lds.coefs[i % 3].co[1][0][0][hb * 32], 2 * kTok, lane % 32);
            wave_fence();
            if ((in & (kStale | 1 << hb)) == 0 && whole(begin + step * 32, 32)) {
                E = choose_range(size);                      // alike in all waves
                in = next_in = kStale;
            }
            // all tiles of rows together (two float32 prompts of 512 tokens, mostly
            // such steps: 46 us, 48 one at a time); with 64 channels one at a time,
            // since the compiler then orders the plain steps better (six bfloat16
            // prompts: 513 us for 551)
            constexpr int kOnce = D == 64 ? 1 : QT;
#pragma unroll
            for (int qt = 0; qt < QT; qt += kOnce) {
                asm volatile("" : "+v"(lane));
                compute(s, lds.coefs[i % 3], hb, begin + step * 32, care_tag, qt, Count<kOnce>{});
            }
        } else {
            compute(s, lds.coefs[i % 3], hb, begin + step * 32, care_tag, 0, Count<QT>{});
        }
    };
    // Careful and plain steps in loops of their own, in the form in which the
    // accumulators are not moved between sets of registers: with 256 channels two
    // loops in turn would move them (45 registers to memory), with fewer a loop in
    // the other one does (2048 float32 rows after 8192 tokens: 800 us for 745).
    if constexpr (D == 256) {
        for (int step = 0; step < steps; ++step) {
            while (plain(step)) {
                advance(step, CareTag<false>{});
                if (++step == steps) break;
            }
            if (step < steps) advance(step, CareTag<true>{});
        }
    } else {
        for (int step = 0; step < steps;) {
            for (; step < steps && !plain(step); ++step) advance(step, CareTag<true>{});
            for (; step < steps && plain(step); ++step) advance(step, CareTag<false>{});
        }
    }
    rows.close();
    rows.write(p, t, kv_head, first_row, lane);
}

}  // namespace qg
