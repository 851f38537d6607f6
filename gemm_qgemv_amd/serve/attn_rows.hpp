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
// 2048 float32 rows after 8192 tokens, 32 heads of 128 channels: 735 us (618
// GFLOP in two pieces, 0.84 PFLOP/s; vector unit 57% and matrix cores 33% busy,
// seldom both). Six bfloat16 prompts of up to 4001 tokens, 32 heads of 64
// channels: 541 us (vector unit 75%: a quarter-rate exponential and 8.5 other
// instructions a score; matrix cores 18%).
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
    float co[2][NG][2][kTok];                              // as in attn_few.hpp
    float top[4];
};

template <int D>
struct RowsLds {
    static constexpr int kRaw = 32 * (D == 64 ? 16 : 32);   // code bytes of V a wave transposes
    RowsTile<D> tile[2];
    uint8_t raw[4][kRaw];
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
    const int64_t first_row = t.row0 + wave * 16 * QT;
    rows.load(p, t, kv_head, first_row, lane);

    // ---- fetching: K block `wave` (mod NB) of the tile, V's codes of 32 tokens
    // and a part of the channels, coefficients of the K block's tokens
    const int32_t *row_pages = p.table + int64_t(t.b) * p.table_stride;
    const int64_t head_off = int64_t(kv_head) * p.kv.block_bytes, half = p.kv.block_bytes >> 1;
    const int page_mask = (1 << p.kv.page_shift) - 1;
    const int k_block = wave % NB, k_group = D == 256 ? wave / NB * KG : 0;
    const int v_half = NH == 2 ? wave >> 1 : 0, v_part = NH == 2 ? wave & 1 : wave;
    int32_t page_ids;
    auto fetch_pages = [&](int tile) {
        const int32_t want = begin + tile * kTok + (lane & (NB - 1)) * 16;
        page_ids = row_pages[(want < end ? want : end - 1) >> p.kv.page_shift];
    };
    u32x2 k_raw[KG];
    uint32_t v_raw[2][VB / 16];
    uint32_t coef[NG];
    auto fetch_tile = [&](int tile) {
        const int32_t base = begin + tile * kTok;
        auto block = [&](int blk, bool &known, int &at) {
            const int32_t id = __builtin_amdgcn_readlane(page_ids, blk);
            known = id >= 0 && id < p.kv.num_pages;
            at = (base + blk * 16) & page_mask;
            return p.kv.data + (known ? id : 0) * p.kv.page_bytes + head_off;
        };
        bool known;
        int at;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint8_t *src = block(v_half * 2 + j, known, at) + half + at * kRow + v_part * VB +
                                 static_cast<uint32_t>((lane >> 2) * kRow + (lane & 3) * (VB / 4));
            if constexpr (VB == 32) {
                const u32x2 v = *reinterpret_cast<const u32x2 *>(src);
                v_raw[j][0] = v[0], v_raw[j][1] = v[1];
            } else {
                v_raw[j][0] = *reinterpret_cast<const uint32_t *>(src);
            }
        }
        const uint8_t *page = block(k_block, known, at);
#pragma unroll
        for (int g = 0; g < KG; ++g)
            k_raw[g] = *reinterpret_cast<const u32x2 *>(page + at * kRow + (k_group + g) * 32 +
                                                        static_cast<uint32_t>((lane & 15) * kRow + (lane >> 4) * 8));
        if (NB == 4 || wave < NB)
            load_coefs(page + ((D / 2) << p.kv.page_shift) + at * (D / 16) +
                           static_cast<uint32_t>(((lane >> 4) & 1) * half + (lane & 15) * (D / 16)),
                       known, base + k_block * 16 + (lane & 15) < end, coef);
    };
    const NibbleBits bits;
    auto put_tile = [&](RowsTile<D> &s) {
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
        if (NB == 4 || wave < NB) {
            float top = 0.0f;
            const bool is_v = (lane >> 4) & 1;
            const float odd = is_v && (lane & 1) ? 0.0625f : 1.0f, centre = is_v && (lane & 1) ? kOddCentre : 8.0f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float sc = __uint_as_float(coef[g] << 16), bi = __uint_as_float(coef[g] & 0xffff0000u);
                top = fmaxf(top, fabsf(sc));
                if (lane < 32) {
                    s.co[is_v][g][0][k_block * 16 + (lane & 15)] = sc * odd;
                    s.co[is_v][g][1][k_block * 16 + (lane & 15)] = kTwo ? fmaf(centre, sc, bi) : bi;
                }
            }
            top = max_over_16(top);
            if (lane == 16) s.top[k_block] = top;            // V's
        }
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

    // ---- 32 tokens: from block 2 hb of the tile on
    auto compute = [&](const RowsTile<D> &s, int hb, float top, int32_t base, auto masked_tag) {
        constexpr bool kMasked = decltype(masked_tag)::value;
        const int g4 = lane >> 4;
        f32x4 x[QT][2];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const f16x8 k0 = __builtin_bit_cast(f16x8, s.k[hb * 2 + a][g][0][lane]);
                const f16x8 k1 = __builtin_bit_cast(f16x8, s.k[hb * 2 + a][g][1][lane]);
                const f32x4 sc = *reinterpret_cast<const f32x4 *>(&s.co[0][g][0][(hb * 2 + a) * 16 + g4 * 4]);
                const f32x4 bi = *reinterpret_cast<const f32x4 *>(&s.co[0][g][1][(hb * 2 + a) * 16 + g4 * 4]);
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) rows.score(qt, g, k0, k1, sc, bi, x[qt][a]);
            }
        uint32_t visible[QT] = {};
#pragma unroll
        for (int qt = 0; qt < QT; ++qt)
            rows.template weigh<kMasked>(p, qt, x[qt], visible[qt], &s.co[1][0][0][hb * 32], 2 * kTok, top, base, g4);
        // small groups of vector and matrix instructions in turn (2048 float32
        // rows after 8192 cached tokens: 735 us, 750 without; with one product a
        // piece, bfloat16, the compiler's own order is as good: 541 and 542)
        if constexpr (kTwo) __builtin_amdgcn_iglp_opt(0);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f16x8 ph[QT], pl[QT];
            f32x4 sc[2], bi[2];
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                sc[a] = *reinterpret_cast<const f32x4 *>(&s.co[1][g][0][(hb * 2 + a) * 16 + g4 * 4]);
                bi[a] = *reinterpret_cast<const f32x4 *>(&s.co[1][g][1][(hb * 2 + a) * 16 + g4 * 4]);
            }
#pragma unroll
            for (int qt = 0; qt < QT; ++qt)
                rows.template pieces<kMasked>(qt, g, x[qt][0], x[qt][1], visible[qt], sc, bi, ph[qt], pl[qt]);
#pragma unroll
            for (int db = 0; db < 4; ++db) {
                const f16x8 v = __builtin_bit_cast(f16x8, s.v[hb][g * 4 + db][lane]);
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) rows.add(qt, g * 4 + db, v, ph[qt], pl[qt]);
            }
        }
    };

    if (tiles > 0) {
        fetch_pages(0);
        fetch_tile(0);
        if (tiles > 1) fetch_pages(1);
    }
    const int steps = (end - begin + 31) / 32;
    auto whole = [&](int step) {
        const int32_t base = begin + step * 32;
        return base + 32 <= end && all_visible(p, t, base, 32);
    };
    auto advance = [&](int step, auto masked_tag) {
        // the lane number is made opaque anew: offsets made from it are then
        // not kept in registers through the loop
        asm volatile("" : "+v"(lane));
        const int i = step / NH, hb = step % NH;
        RowsTile<D> &s = lds.tile[i & 1];
        if (hb == 0) {
            put_tile(s);
            __syncthreads();
            if (i + 1 < tiles) {
                fetch_tile(i + 1);
                if (i + 2 < tiles) fetch_pages(i + 2);
            }
        }
        compute(s, hb, fmaxf(s.top[2 * hb], s.top[2 * hb + 1]), begin + step * 32, masked_tag);
    };
    // a loop for steps that need masks and one for those that do not (one loop
    // with both in it moves the accumulators between two sets of registers)
    for (int step = 0; step < steps;) {
        for (; step < steps && !whole(step); ++step) advance(step, MaskTag<true>{});
        for (; step < steps && whole(step); ++step) advance(step, MaskTag<false>{});
    }
    rows.close();
    rows.write(p, t, kv_head, first_row, lane);
}

}  // namespace qg
