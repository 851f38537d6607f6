// attn_few.hpp -- attention for few query rows of a request and key/value
// head (up to 16 RW): decode steps and checks of a few speculated tokens.
//
// The four waves of a workgroup are RW groups of 16 rows times KW = 4 / RW
// groups that take tiles of tokens in turn. A tile's codes are fetched into
// registers one tile ahead and passed through LDS; with RW = 1 a wave passes
// its own tile to itself and waits for no other. The KW partial results meet
// in LDS at the end. Careful tiles (attn_common.hpp) go through 32 tokens at a time.
//
// 16 rows are the least a matrix instruction takes: with 4 query heads a
// key/value head 12 columns are idle, and the vector work of a tile (600
// instructions of 64 tokens at 128 channels in float32, half of them to make
// operands of the codes) is the same for 1 row as for 16. With the join: 64
// bfloat16 requests of 1024 to 8192 tokens (360 MB) 90 us, 4.0 TB/s, all of it
// from one page 71, so part memory, most the waves' own chains; one float32
// request of 131071 (151 MB) 45 us, 3.4 TB/s, from one page 42: the chains, at two
// waves a SIMD.
#pragma once

#include "attn_common.hpp"

namespace qg {

// Tokens of a tile: 64, or 32 where the accumulators and query operands of a
// wave leave no registers for the scores of 64.
constexpr int few_tile_tokens(int dim) { return dim == 256 ? 32 : 64; }

// Granule (16-byte piece of a token's codes) t is stored at, so that the 16
// lanes of a read fall on different banks: K is read 16 consecutive tokens at
// a time, V the tokens 16 a + 4 g4 + i.
template <int D>
__device__ __forceinline__ int k_swizzle(int t)
{
    return D == 64 ? (t >> 3) & 1 : D == 128 ? (t >> 2) & 3 : (t >> 1) & 7;
}
template <int D>
__device__ __forceinline__ int v_swizzle(int t)
{
    return D == 64 ? (t >> 4) & 1 : D == 128 ? (t >> 4) & 3 : ((t >> 1) & 1) | (((t >> 4) & 3) << 1);
}

// LDS of one group of waves: a tile's codes and its coefficients as float32.
template <int D, int TOK>
struct TileLds {
    static constexpr int kTok = TOK;
    static constexpr int kRow = D / 2;                     // code bytes of a token
    uint8_t codes[2 * kTok * kRow];                        // K, V
    // scale (V, odd tokens: / 16) and bias (float32 queries: + centre * scale) of K, V
    float co[2][D / 64][2][kTok];
};

// Bytes of LDS a workgroup needs for tiles (and for the join), and in all.
template <int D>
constexpr int few_tiles_bytes()
{
    // RW = 1: a tile for each wave; RW = 2: two buffers for each pair of waves
    const int tiles = static_cast<int>(sizeof(TileLds<D, few_tile_tokens(D)>)) * 4;
    const int join = 4 * 16 * (D + 4) * 4;
    return tiles > join ? tiles : join;
}
template <int D>
constexpr int few_lds_bytes()
{
    // and, for careful tiles, each wave's notes of a tile and its rows' tokens
    return few_tiles_bytes<D>() + 4 * static_cast<int>(sizeof(TileSizes) + 16 * sizeof(int32_t));
}

// Three workgroups a compute unit (168 registers) up to 128 channels, two
// beyond: 64 requests of up to 8192 tokens, 128 channels: float32 125 us at two,
// 106 at three, bfloat16 89.6 and 89.5.
template <typename T, int D, int RW>
__global__ __launch_bounds__(kAttnThreads, D == 256 ? 2 : 3) void attn_few_kernel(AttnParams p)
{
    constexpr int KW = 4 / RW;                             // groups of waves that share out the tokens
    constexpr bool kTwo = sizeof(T) == 4;                  // float32: two pieces
    constexpr int kTok = few_tile_tokens(D), NG = D / 64;
    constexpr int R = 16 * RW;                             // query rows of the workgroup
    constexpr int kRow = D / 2, kSeg = kRow / 16;          // code bytes, 16-byte granules of a token
    extern __shared__ __align__(16) uint8_t lds[];

    // the lane number is made opaque anew in every round of tiles: the many
    // LDS and memory offsets made from it are then computed where they are
    // used instead of being kept in registers through the loop
    int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rw = wave % RW, kw = wave / RW;
    int col = lane & 15, g4 = lane >> 4;
    const int kv_head = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.kv.heads));
    RowTile t;
    if (!find_tile<R>(p, blockIdx.x / static_cast<unsigned>(p.kv.heads), t)) return;

    int32_t begin, end;
    if (!split_tokens(p, t, kTok, begin, end)) return;
    const int tiles = (end - begin + kTok - 1) / kTok;

    QueryRows<T, D, 1> rows;
    const uint32_t first_row = t.row0 + rw * 16;
    TileSizes &sizes = reinterpret_cast<TileSizes *>(lds + few_tiles_bytes<D>())[wave];
    int32_t *const pos = reinterpret_cast<int32_t *>(lds + few_tiles_bytes<D>() + 4 * sizeof(TileSizes)) + wave * 16;
    rows.load(p, t, kv_head, first_row, lane, pos);

    // ---- fetching tiles -----------------------------------------------------
    const int32_t *row_pages = p.table + int64_t(t.b) * p.table_stride;
    const int64_t head_off = int64_t(kv_head) * p.kv.block_bytes;
    const int page_mask = (1 << p.kv.page_shift) - 1;
    using Tile = TileLds<D, kTok>;
    Tile *const bufs = reinterpret_cast<Tile *>(lds) + kw * (RW > 1 ? 2 : 1);

    // A tile comes in blocks of 16 tokens (a page holds whole blocks), which a
    // wave reads as contiguous pieces: the block's address is scalar, a lane's
    // offset constant. The waves of a group take blocks in turn.
    constexpr int NB = kTok / 16, NBW = NB / RW;
    constexpr int kPieces = D == 64 ? 1 : 2 * (D / 128);    // 16-byte loads a lane makes for a block
    const int64_t half = p.kv.block_bytes >> 1;
    // part (K 0, V 1), token in the block and granule of a lane's piece n
    auto piece_part = [&](int n) { return D == 64 ? lane >> 5 : n / (D / 128); };
    auto piece_token = [&](int n) { return D == 64 ? (lane & 31) >> 1 : (n % (D / 128)) * (64 / kSeg) + lane / kSeg; };
    int32_t page_ids;                                       // lane j: the page of block j (mod NB)
    auto fetch_pages = [&](int tile) {
        const int32_t want = begin + tile * kTok + (lane & (NB - 1)) * 16;
        page_ids = row_pages[(want < end ? want : end - 1) >> p.kv.page_shift];
    };
    u32x4 code[NBW][kPieces];
    uint32_t coef[NB][NG];                                  // lane: part (lane / 16) % 2, token lane % 16; of all blocks
    int unknown = 0;                                        // bits: blocks whose page is outside the cache
    auto fetch_tile = [&](int tile) __attribute__((always_inline)) {
        const int32_t base = begin + tile * kTok;
        unknown = 0;
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
            const int32_t id = __builtin_amdgcn_readlane(page_ids, blk);
            const bool known = static_cast<uint32_t>(id) < static_cast<uint32_t>(p.kv.num_pages);
            const uint8_t *page = p.kv.data + (known ? id : 0) * p.kv.page_bytes + head_off;
            const int at = (base + blk * 16) & page_mask;
            load_coefs(page + ((D / 2) << p.kv.page_shift) + at * (D / 16) +
                           static_cast<uint32_t>(((lane >> 4) & 1) * half + (lane & 15) * (D / 16)),
                       coef[blk]);
            unknown |= known ? 0 : 1 << blk;
        }
#pragma unroll
        for (int j = 0; j < NBW; ++j) {
            const int blk = rw + j * RW;
            const int32_t id = __builtin_amdgcn_readlane(page_ids, blk);
            const bool known = static_cast<uint32_t>(id) < static_cast<uint32_t>(p.kv.num_pages);
            const uint8_t *page = p.kv.data + (known ? id : 0) * p.kv.page_bytes + head_off;
            const int at = (base + blk * 16) & page_mask;
            const uint8_t *src = page + at * kRow;
#pragma unroll
            for (int n = 0; n < kPieces; ++n) {
                if constexpr (D == 64)
                    code[j][n] = *reinterpret_cast<const u32x4 *>(src + static_cast<uint32_t>((lane >> 5) * half + (lane & 31) * 16));
                else
                    code[j][n] = *reinterpret_cast<const u32x4 *>(src + piece_part(n) * half + (n % (D / 128)) * 1024 +
                                                                  static_cast<uint32_t>(lane * 16));
            }
        }
    };
    // the fetched tile into LDS (a plain one is known, and the request's, throughout)
    auto put_tile = [&](Tile &s, int32_t base, auto care_tag) __attribute__((always_inline)) {
        const bool is_v = (lane >> 4) & 1;
        const float odd = is_v && (lane & 1) ? 0.0625f : 1.0f, centre = is_v && (lane & 1) ? kOddCentre : 8.0f;
#pragma unroll
        for (int j = 0; j < NBW; ++j) {
            const int blk = rw + j * RW;
#pragma unroll
            for (int n = 0; n < kPieces; ++n) {
                const int part = piece_part(n), tok = blk * 16 + piece_token(n), seg = lane % kSeg;
                const int to = seg ^ (part == 0 ? k_swizzle<D>(tok) : v_swizzle<D>(tok));
                *reinterpret_cast<u32x4 *>(s.codes + (part * kTok + tok) * kRow + to * 16) = code[j][n];
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t c = RW == 1 ? coef[j][g] : rw ? coef[j * RW + RW - 1][g] : coef[j * RW][g];
                if constexpr (decltype(care_tag)::value) c = coef_of(c, (unknown >> blk & 1) == 0, base + blk * 16 + (lane & 15) < end);
                const float sc = __uint_as_float(c << 16), bi = __uint_as_float(c & 0xffff0000u);
                if (lane < 32) {
                    s.co[is_v][g][0][blk * 16 + (lane & 15)] = sc * odd;
                    s.co[is_v][g][1][blk * 16 + (lane & 15)] = kTwo ? fmaf(centre, sc, bi) : bi;
                }
            }
        }
    };

    int E = kAbove;                                         // range of plain tiles' value scales, up to 4 at first
    const NibbleBits bits;
    // ---- TOKENS tokens of a tile, from block `first` on ---------------------
    auto compute = [&](const Tile &s, int first, int32_t base, auto care_tag, auto tokens_tag) __attribute__((always_inline)) {
        constexpr bool kCareful = decltype(care_tag)::value;
        constexpr int kTokens = decltype(tokens_tag)::value, NA = kTokens / 16, NST = kTokens / 32;
        f32x4 x[NA];
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            const int tok = (first + a) * 16 + col;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int seg = (g * 2 + (g4 >> 1)) ^ k_swizzle<D>(tok);
                const u32x2 w = *reinterpret_cast<const u32x2 *>(s.codes + tok * kRow + seg * 16 + (g4 & 1) * 8);
                rows.score(0, g, nibbles<kTwo>(w[0], bits), nibbles<kTwo>(w[1], bits),
                           *reinterpret_cast<const f32x4 *>(&s.co[0][g][0][(first + a) * 16 + g4 * 4]),
                           *reinterpret_cast<const f32x4 *>(&s.co[0][g][1][(first + a) * 16 + g4 * 4]), x[a]);
            }
        }
        uint32_t visible = 0;
        rows.template weigh<kCareful>(p, 0, kCareful ? pos[col] : 0, x, visible, &sizes, first * 16, E, base + first * 16, g4);
        // out += V^T w: lane `col` of group g4 addresses the codes of token
        // 16 (col / 4) + 4 g4 + col % 4 and gets channel `col` of 16 tokens
        // (32-token tiles: of 8 tokens for each of two blocks of channels)
        constexpr int kBlocks = kTok == 64 ? 1 : 2;          // blocks of 16 channels a read serves
        const int v_tok = kTok == 64 ? (col >> 2) * 16 + g4 * 4 + (col & 3) : ((col >> 2) & 1) * 16 + g4 * 4 + (col & 3);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            __builtin_amdgcn_sched_barrier(0);               // or the operands of several groups are held at once
            f16x8 ph[NST], pl[NST];
            float down = 1.0f;
#pragma unroll
            for (int st = 0; st < NST; ++st) {
                f32x4 sc[2], bi[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sc[h] = *reinterpret_cast<const f32x4 *>(&s.co[1][g][0][(first + st * 2 + h) * 16 + g4 * 4]);
                    bi[h] = *reinterpret_cast<const f32x4 *>(&s.co[1][g][1][(first + st * 2 + h) * 16 + g4 * 4]);
                }
                rows.template pieces<kCareful>(0, g, x[st * 2], x[st * 2 + 1], visible >> (st * 8), sc, bi, ph[st], pl[st], down);
            }
#pragma unroll
            for (int n = 0; n < 4 / kBlocks; ++n) {
                const int chunk = g * 4 + n * kBlocks + (kBlocks == 2 ? col >> 3 : 0);
                const int seg = (chunk >> 1) ^ v_swizzle<D>(v_tok);
                const i32x2 w = read_transposed(s.codes + (kTok + v_tok) * kRow + seg * 16 + (chunk & 1) * 8);
                auto operand = [&](int h) { return nibbles<kTwo, kOddCentre>(static_cast<uint32_t>(h ? w[1] : w[0]), bits); };
                if constexpr (kBlocks == 2) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const f16x8 v[1] = {operand(h)};
                        rows.template add<kCareful>(0, g * 4 + n * 2 + h, v, ph, pl, down);
                    }
                } else if constexpr (kTokens == 64) {
                    const f16x8 v[2] = {operand(0), operand(1)};
                    rows.template add<kCareful>(0, g * 4 + n, v, ph, pl, down);
                } else {
                    const f16x8 v[1] = {operand(first / 2)};
                    rows.template add<kCareful>(0, g * 4 + n, v, ph, pl, down);
                }
            }
        }
    };

    const int trips = (tiles + KW - 1) / KW;
    if (kw < tiles) {
        fetch_pages(kw);
        fetch_tile(kw);
        if (kw + KW < tiles) fetch_pages(kw + KW);
    }
    // whether round i's tile needs no care: every row sees all of its tokens, and
    // the value scales (of the fetched tile; lanes of V) are in the range
    auto whole = [&](int i) {
        const int32_t base = begin + (kw + i * KW) * kTok;
        return base + kTok <= end && all_visible(p, t, base, kTok);
    };
    auto plain = [&](int i) {
        if (unknown != 0 || !whole(i)) return false;
        bool in = true;
#pragma unroll
        for (int blk = 0; blk < NB; ++blk)
#pragma unroll
            for (int g = 0; g < NG; ++g) in = in & in_range(coef[blk][g], E);
        return (__ballot(in) >> 16 & 0xffff) == 0xffff;
    };
    auto advance = [&](int i, auto care_tag) __attribute__((always_inline)) {
        const int tile = kw + i * KW;
        const bool live = tile < tiles;
        asm volatile("" : "+v"(lane));
        col = lane & 15, g4 = lane >> 4;
        Tile &s = bufs[RW > 1 ? i & 1 : 0];
        if (live) put_tile(s, begin + tile * kTok, care_tag);
        if constexpr (RW > 1) __syncthreads();
        else wave_fence();
        if (!live) return;
        if constexpr (decltype(care_tag)::value) {
            const float size = note_sizes<NG>(sizes, &s.co[1][0][0][0], 2 * kTok, lane % kTok);
            wave_fence();
            if (whole(i)) E = choose_range(size);            // alike in the waves that share the tile
        }
        if (tile + KW < tiles) {
            fetch_tile(tile + KW);
            if (tile + 2 * KW < tiles) fetch_pages(tile + 2 * KW);
        }
        if constexpr (decltype(care_tag)::value) {
            // 32 tokens at a time, which need fewer registers
#pragma unroll
            for (int first = 0; first < kTok / 16; first += 2) {
                asm volatile("" : "+v"(lane));
                col = lane & 15, g4 = lane >> 4;
                compute(s, first, begin + tile * kTok, care_tag, Count<32>{});
            }
        } else {
            compute(s, 0, begin + tile * kTok, care_tag, Count<kTok>{});
        }
        if constexpr (RW == 1) wave_fence();
    };
    // plain tiles in a loop of their own (as one of two loops, or in one with the
    // careful tiles, the accumulators are moved between sets of registers); either
    // has one barrier a round, so waves may be in different ones
    for (int i = 0; i < trips; ++i) {
        while (plain(i)) {
            advance(i, CareTag<false>{});
            if (++i == trips) break;
        }
        if (i < trips) advance(i, CareTag<true>{});
    }

    // ---- the groups of waves joined --------------------------------------------
    rows.close();
    constexpr int kPitch = D + 4;
    __syncthreads();                                       // every wave is done with its tiles
    float *mine = reinterpret_cast<float *>(lds) + (rw * KW + kw) * 16 * kPitch + col * kPitch;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) *reinterpret_cast<f32x4 *>(mine + d * 16 + g4 * 4) = rows.acc[0][d];
    if (g4 == 0) mine[D] = rows.ref[0], mine[D + 1] = rows.total[0];
    __syncthreads();
    // the KW waves of a row group share its rows; 4 channels a thread
    const float *all = reinterpret_cast<const float *>(lds) + rw * KW * 16 * kPitch;
    constexpr int kQuads = D / 4;
    uint32_t group = p.group;
    asm volatile("" : "+s"(group));                        // or its reciprocal stays in a register from load() on
    for (int i = kw * 64 + lane; i < 16 * kQuads; i += KW * 64) {
        const int r = i / kQuads, d = (i % kQuads) * 4;
        const uint32_t row = first_row + r;
        if (row >= t.rows) continue;
        float m = kNoReference, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            const float rf = all[(w * 16 + r) * kPitch + D];
            m = rf > m || rf != rf ? rf : m;
        }
        f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            const float *src = all + (w * 16 + r) * kPitch;
            const float f = __builtin_amdgcn_exp2f(src[D] - m);
            sum = fmaf(f, src[D + 1], sum);
            o += f * *reinterpret_cast<const f32x4 *>(src + d);
        }
        const uint32_t tok = row / group;
        const int head = kv_head * p.group + static_cast<int>(row - tok * group);
        const int64_t orow = int64_t(t.q0 + tok) * p.q_heads + head;
        if (p.nsplit > 1) {
            const int64_t at = orow * p.nsplit + blockIdx.y;
            *reinterpret_cast<f32x4 *>(p.part_out + at * D + d) = o;
            if (d == 0) p.part_stat[at * 2] = m, p.part_stat[at * 2 + 1] = sum;
        } else {
            store_out4(static_cast<T *>(p.out) + int64_t(t.q0 + tok) * p.out_stride + int64_t(head) * D + d, o * attn_inverse(t, sum));
            if (p.lse && d == 0) p.lse[orow] = attn_lse(t, m, sum);
        }
    }
}

}  // namespace qg
