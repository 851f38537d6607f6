// attn.hpp -- causal attention of new tokens over the paged 4-bit cache.
//
// Mathematics. For a query row q and tokens t with key k_t[d] =
// s_t[g] * c_t[d] + b_t[g] (g = d / 64, c the 4-bit code),
//
//   x_t = q . k_t = sum_g ( s_t[g] * sum_{d in g} q[d] c_t[d] + b_t[g] * Q[g] ),   Q[g] = sum_{d in g} q[d],
//   out[d] = ( sum_t (w_t s'_t[g]) (c'_t[d] - 8) + sum_t w_t (b'_t[g] + 8 s'_t[g]) ) / sum_t w_t,   w_t = 2^(f x_t - R),
//
// one pass over the tokens with a reference R a row (the softmax does not
// depend on R). The codes themselves go to the matrix cores: they are exact
// in binary16, so nothing of the cache is rounded, and a float32 query or
// weight goes as two binary16 pieces (22 bits) where a dequantized cache
// would need three products of pieces. Scales and biases are applied in
// float32 outside of them. The value codes are centred (c - 8) so that the
// accumulators hold sums that cancel no worse than the result does.
//
// Operand layouts (v_mfma_f32_16x16x32_f16; l = lane, g4 = l / 16):
//   scores   A = 16 tokens (row l % 16) x 32 channels, B = 32 channels x 16
//            query rows (column l % 16), C = lane holds tokens 4 g4 + 0..3 of
//            query row l % 16;
//   output   A = 16 channels x 32 tokens (V transposed), B = 32 tokens x 16
//            query rows, C = lane holds channels 4 g4 + 0..3 of row l % 16.
// The order of the contracted index is free as long as A and B agree. So a
// lane's score results are its B operand of the second product as they are
// (no exchange between lanes), and the nibbles of a dword are masked in
// place: halves (n, n + 4) of a dword come out of one AND, as binary16
// subnormals n * 2^-24 (K) or, with an OR and a packed add, as c - 8 (V); odd
// nibbles come out 16 times too large, which the other operand makes good.
// V's codes are stored token by token; ds_read_b64_tr_b4 transposes 16 x 16
// nibbles among 16 lanes as it reads them.
//
// Work. A workgroup has 4 waves as RW groups of 16 * QT query rows (of one
// request and key/value head: the heads that share it, and its new tokens,
// are rows alike) times KW groups that take tiles of kTok tokens in turn. A
// tile's codes are fetched into registers one tile ahead and passed through
// LDS; with RW = 1 a wave passes its own tile to itself and waits for no
// other. Tokens are cut into `nsplit` chunks over workgroups where rows are
// few; partial results (reference, sum, output) are joined by
// attn_join_kernel in a fixed order.
#pragma once

#include "kv_cache.hpp"

namespace qg {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct AttnParams {
    const void *q;
    int64_t q_stride;
    KvView kv;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *cu_q, *kv_len;
    int batch;
    int64_t total_q;
    int32_t max_kv;
    int group;            // query heads of one key/value head
    int q_heads;
    float scale_log2e;
    int64_t window;       // 0: none
    void *out;
    int64_t out_stride;
    float *lse;
    float *part_out;      // [total_q * q_heads][nsplit][D]
    float *part_stat;     // [total_q * q_heads][nsplit][2]: reference, sum
    int nsplit;
    int32_t chunk;        // tokens of a split (a multiple of the tile of a workgroup)
};

constexpr int kAttnThreads = 256;
constexpr float kNoReference = -1e30f;   // below every score; finite, so that differences stay defined
// A weight times a value scale stays below 2^(kHead + kSlack) in binary16;
// the reference moves only when a score passes it by kSlack, so the
// accumulators are rarely rescaled.
constexpr float kHead = 7.0f, kSlack = 7.0f;

// Tokens of a tile: 64, or 32 where the accumulators and query operands of a
// wave (D * QT) leave no registers for the scores of 64.
constexpr int attn_tile_tokens(int dim, int qt) { return dim * qt >= 256 ? 32 : 64; }

// The rows of one tile of query rows: request b, rows row0.. of its rows
// (row = token * group + head), and the tokens [lo, hi) that any of them sees.
struct RowTile {
    int b;
    int32_t q0;           // first query row of the request in the batch
    int32_t n_q, kv;      // its new tokens and its tokens
    int64_t row0, rows;
    int32_t lo, hi;
    bool poison;          // longer than the call allows
};

__device__ __forceinline__ int32_t attn_cu(const AttnParams &p, int b)
{
    const int64_t v = p.cu_q[b];
    return static_cast<int32_t>(v < 0 ? 0 : v > p.total_q ? p.total_q : v);
}

// Tile slots are dealt to requests without their exact tile counts:
// request b starts at slot floor(cu_q[b] * group / R) + b, which leaves room
// for ceil(rows / R) tiles; slots in between are empty.
template <int R>
__device__ __forceinline__ int64_t tile_start(const AttnParams &p, int b)
{
    return int64_t(attn_cu(p, b)) * p.group / R + b;
}

__device__ __forceinline__ void tile_tokens(const AttnParams &p, RowTile &t, int64_t row0, int R)
{
    t.kv = p.kv_len[t.b] < 0 ? 0 : p.kv_len[t.b];
    t.poison = t.kv > p.max_kv;
    if (t.poison) t.kv = 0;
    t.row0 = row0;
    t.rows = int64_t(t.n_q) * p.group;
    const int64_t last = row0 + R < t.rows ? row0 + R : t.rows;
    const int64_t first_pos = int64_t(t.kv) - t.n_q + row0 / p.group;
    const int64_t last_pos = int64_t(t.kv) - t.n_q + (last - 1) / p.group;
    t.hi = last_pos < 0 ? 0 : static_cast<int32_t>(last_pos + 1);
    const int64_t lo = p.window > 0 ? first_pos - p.window + 1 : 0;
    t.lo = lo < 0 ? 0 : lo < t.hi ? static_cast<int32_t>(lo) : t.hi;
}

template <int R>
__device__ __forceinline__ bool find_tile(const AttnParams &p, int64_t slot, RowTile &t)
{
    const int lane = threadIdx.x & 63;
    int count = 0;
    for (int base = 0; base < p.batch; base += 64) {
        const int b = base + lane;
        const uint64_t m = __ballot(b < p.batch && tile_start<R>(p, b) <= slot);
        count += __popcll(m);
        if (m != ~0ull) break;
    }
    if (count == 0) return false;
    t.b = count - 1;
    t.q0 = attn_cu(p, t.b);
    t.n_q = attn_cu(p, t.b + 1) - t.q0;
    const int64_t row0 = (slot - tile_start<R>(p, t.b)) * R;
    if (t.n_q <= 0 || row0 >= int64_t(t.n_q) * p.group) return false;
    tile_tokens(p, t, row0, R);
    return true;
}

// Eight nibbles of a dword as binary16 subnormals: halves (0,4), (1,5)*16,
// (2,6), (3,7)*16, each times 2^-24.
__device__ __forceinline__ f16x8 nibbles_tiny(uint32_t w)
{
    const uint32_t v = w >> 8;
    const u32x4 r = {w & 0x000f000fu, w & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u};
    return __builtin_bit_cast(f16x8, r);
}

// Masks and the bits of 1024 in registers: an AND and an OR with two literals
// would not go into one instruction.
struct NibbleBits {
    uint32_t even = 0x000f000fu, odd = 0x00f000f0u, thousand = 0x64006400u;
    __device__ NibbleBits() { asm("" : "+s"(even), "+s"(odd), "+v"(thousand)); }
};

// Eight nibbles as c - 8: halves (0,4), (1,5)*16, (2,6), (3,7)*16. With the
// bits of 1024 set, a half is 1024 + nibble (or + 16 nibble) exactly.
__device__ __forceinline__ f16x8 nibbles_centred(uint32_t w, const NibbleBits &k)
{
    const uint32_t v = w >> 8;
    const f16x2 even = {(_Float16)-1032.0f, (_Float16)-1032.0f}, odd = {(_Float16)-1152.0f, (_Float16)-1152.0f};
    auto put = [&](uint32_t x, uint32_t mask, f16x2 off) {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (x & mask) | k.thousand) + off);
    };
    const u32x4 r = {put(w, k.even, even), put(w, k.odd, odd), put(v, k.even, even), put(v, k.odd, odd)};
    return __builtin_bit_cast(f16x8, r);
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b)
{
    const f16x2 h = {static_cast<_Float16>(a), static_cast<_Float16>(b)};
    uint32_t v = __builtin_bit_cast(uint32_t, h);
    // A remainder is taken against these bits: without this the compiler
    // rounds a product twice, fused to binary16 for the remainder and by way
    // of float32 for the pair, and one of some 8000 pairs differs.
    asm("" : "+v"(v));
    return v;
}

// A dword of codes as an operand. With float32 queries the codes are centred;
// the matrix cores take subnormals, but keep fewer bits of sums of their
// products (scores 5 times, outputs 8 times as far from the exact ones), which
// bfloat16's own rounding covers, at 5 instead of 9 instructions a dword.
template <bool CENTRED>
__device__ __forceinline__ f16x8 nibbles(uint32_t w, const NibbleBits &k)
{
    if constexpr (CENTRED) return nibbles_centred(w, k);
    else return nibbles_tiny(w);
}

// Maximum (NaN ignored) over the four lanes that share l % 16.
__device__ __forceinline__ float max_over_groups(float v)
{
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

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
    // scale (V, odd tokens: / 16) and bias (float32 queries: + 8 scale) of K, V
    float co[2][D / 64][2][kTok];
    float top[4];                                          // largest |value scale| of a staging wave
};

// bytes of LDS a workgroup needs
template <int D, int RW, int KW, int QT>
constexpr int attn_lds_bytes()
{
    const int tiles = static_cast<int>(sizeof(TileLds<D, attn_tile_tokens(D, QT)>)) * KW * (RW > 1 ? 2 : 1);
    const int join = KW > 1 ? RW * KW * 16 * QT * (D + 4) * 4 : 0;
    return tiles > join ? tiles : join;
}

template <typename T>
__device__ __forceinline__ void store_out4(T *dst, f32x4 v);
template <>
__device__ __forceinline__ void store_out4<float>(float *dst, f32x4 v) { *reinterpret_cast<f32x4 *>(dst) = v; }
template <>
__device__ __forceinline__ void store_out4<uint16_t>(uint16_t *dst, f32x4 v)
{
    u32x2 w = {f32_to_bf16_bits(v[0]) | (f32_to_bf16_bits(v[1]) << 16), f32_to_bf16_bits(v[2]) | (f32_to_bf16_bits(v[3]) << 16)};
    *reinterpret_cast<u32x2 *>(dst) = w;
}

template <bool MASKED>
struct MaskTag {
    static constexpr bool value = MASKED;
};

template <typename T, int D, int RW, int KW, int QT>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_kernel(AttnParams p)
{
    static_assert(RW * KW * 64 == kAttnThreads, "four waves");
    constexpr bool kTwo = sizeof(T) == 4;                  // float32: two pieces
    constexpr int kTok = attn_tile_tokens(D, QT), NA = kTok / 16, NST = kTok / 32, NG = D / 64;
    constexpr float kUnit = kTwo ? 1.0f : 5.9604644775390625e-08f;       // of a code as the matrix cores see it
    constexpr int R = 16 * QT * RW;                        // query rows of the workgroup
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

    // this split's tokens
    const int32_t from = t.lo / kTok * kTok;
    const int64_t b64 = int64_t(from) + int64_t(blockIdx.y) * p.chunk;
    const int32_t begin = b64 < t.hi ? static_cast<int32_t>(b64) : t.hi;
    const int32_t end = t.hi - begin < p.chunk ? t.hi : begin + p.chunk;
    if (begin >= end && blockIdx.y > 0) return;
    const int tiles = (end - begin + kTok - 1) / kTok;

    // ---- the query rows of this wave, as B operands -------------------------
    f16x8 qh[QT][NG][2], ql[kTwo ? QT : 1][NG][2];
    float qsum[QT][NG], factor[QT];
    int32_t pos[QT];                                       // the row's token, -1 for no row
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        const int64_t row = t.row0 + rw * 16 * QT + qt * 16 + col;
        const bool live = row < t.rows;
        const int32_t tok = live ? static_cast<int32_t>(row / p.group) : 0;
        const int head = kv_head * p.group + (live ? static_cast<int>(row - int64_t(tok) * p.group) : 0);
        pos[qt] = live ? t.kv - t.n_q + tok : -1;
        const T *src = static_cast<const T *>(p.q) + int64_t(t.q0 + tok) * p.q_stride + int64_t(head) * D;
        float x[NG][2][8];
        float top = 0.0f;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                load8(src + g * 64 + g4 * 16 + st * 8, x[g][st]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[g][st][i] = live ? x[g][st][i] : 0.0f;
                    top = fmaxf(top, fabsf(x[g][st][i]));
                }
            }
        top = max_over_groups(top);
        // power of two that brings the row's largest element into [2^13, 2^14)
        int e = static_cast<int>((__float_as_uint(top) >> 23) & 0xff);
        e = e < 40 ? 40 : e > 240 ? 240 : e;
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 13 + 127 - e) << 23);
        // scores come out as (q * up) . (code * kUnit)
        factor[qt] = p.scale_log2e / kUnit * __uint_as_float(static_cast<uint32_t>(127 - 13 - 127 + e) << 23);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float sum = 0.0f;
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                u32x4 h, l;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float a = x[g][st][r] * up, b = x[g][st][r + 4] * up;
                    sum += a + b;
                    const float sa = r & 1 ? a * 0.0625f : a, sb = r & 1 ? b * 0.0625f : b;
                    const uint32_t pair = pack_f16(sa, sb);
                    const f16x2 hh = __builtin_bit_cast(f16x2, pair);
                    h[r] = pair;
                    l[r] = pack_f16(sa - static_cast<float>(hh[0]), sb - static_cast<float>(hh[1]));
                }
                qh[qt][g][st] = __builtin_bit_cast(f16x8, h);
                if constexpr (kTwo) ql[qt][g][st] = __builtin_bit_cast(f16x8, l);
            }
            sum = pair_sum<5>(pair_sum<4>(sum));
            qsum[qt][g] = sum * kUnit;
        }
    }

    f32x4 acc[QT][D / 16];
    float ref[QT], total[QT], bias[QT][NG];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        ref[qt] = kNoReference;
        total[qt] = 0.0f;
#pragma unroll
        for (int g = 0; g < NG; ++g) bias[qt][g] = 0.0f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) acc[qt][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // ---- fetching tiles -----------------------------------------------------
    const int32_t *row_pages = p.table + int64_t(t.b) * p.table_stride;
    const int64_t head_off = int64_t(kv_head) * p.kv.block_bytes;
    const int page_mask = (1 << p.kv.page_shift) - 1;
    using Tile = TileLds<D, kTok>;
    Tile *const bufs = reinterpret_cast<Tile *>(lds) + kw * (RW > 1 ? 2 : 1);

    // A tile comes in blocks of 16 tokens (a page holds whole blocks), which a
    // wave reads as contiguous pieces: the block's address is scalar, a lane's
    // offset constant. The waves of a group take blocks in turn; with more
    // waves than blocks K and V of a block go to two of them.
    constexpr int NB = kTok / 16, NBW = RW < NB ? NB / RW : 1;
    constexpr bool kHalves = RW > NB;
    constexpr int kPieces = D == 64 ? 1 : (kHalves ? 1 : 2) * (D / 128);     // 16-byte loads a lane makes for a block
    const int my_block = rw % NB, my_part = kHalves ? rw / NB : 0;
    const int64_t half = p.kv.block_bytes >> 1;
    // part (K 0, V 1), token in the block and granule of a lane's piece n
    auto piece_part = [&](int n) { return D == 64 ? lane >> 5 : kHalves ? my_part : n / (D / 128); };
    auto piece_token = [&](int n) { return D == 64 ? (lane & 31) >> 1 : (n % (D / 128)) * (64 / kSeg) + lane / kSeg; };
    int32_t page_ids;                                       // lane j: the page of block j (mod NB)
    auto fetch_pages = [&](int tile) {
        const int32_t want = begin + tile * kTok + (lane & (NB - 1)) * 16;
        page_ids = row_pages[(want < end ? want : end - 1) >> p.kv.page_shift];
    };
    u32x4 code[NBW][kPieces];
    uint32_t coef[NBW][NG];                                 // lane: part (lane / 16) % 2, token lane % 16
    auto fetch_tile = [&](int tile) {
        const int32_t base = begin + tile * kTok;
#pragma unroll
        for (int j = 0; j < NBW; ++j) {
            const int blk = my_block + j * RW;
            const int32_t id = __builtin_amdgcn_readlane(page_ids, blk);
            const bool known = id >= 0 && id < p.kv.num_pages;
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
            if (!kHalves || my_part == 0) {
                const uint8_t *co = page + ((D / 2) << p.kv.page_shift) + at * (D / 16) +
                                    static_cast<uint32_t>(((lane >> 4) & 1) * half + (lane & 15) * (D / 16));
                if constexpr (NG == 1) {
                    coef[j][0] = *reinterpret_cast<const uint32_t *>(co);
                } else if constexpr (NG == 2) {
                    const u32x2 v = *reinterpret_cast<const u32x2 *>(co);
                    coef[j][0] = v[0], coef[j][1] = v[1];
                } else {
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(co);
#pragma unroll
                    for (int g = 0; g < NG; ++g) coef[j][g] = v[g];
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    if (!known) coef[j][g] = 0x7fc07fc0u;                              // a page outside the cache reads as NaN
                    if (base + blk * 16 + (lane & 15) >= end) coef[j][g] = 0;          // places behind the last token hold anything
                }
            }
        }
    };
    // the fetched tile into LDS; returns the largest |value scale| this wave saw
    auto put_tile = [&](Tile &s) {
        float top = 0.0f;
        const bool is_v = (lane >> 4) & 1;
        const float odd = is_v && (lane & 1) ? 0.0625f : 1.0f;
#pragma unroll
        for (int j = 0; j < NBW; ++j) {
            const int blk = my_block + j * RW;
#pragma unroll
            for (int n = 0; n < kPieces; ++n) {
                const int part = piece_part(n), tok = blk * 16 + piece_token(n), seg = lane % kSeg;
                const int to = seg ^ (part == 0 ? k_swizzle<D>(tok) : v_swizzle<D>(tok));
                *reinterpret_cast<u32x4 *>(s.codes + (part * kTok + tok) * kRow + to * 16) = code[j][n];
            }
            if (!kHalves || my_part == 0) {
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float sc = __uint_as_float(coef[j][g] << 16), bi = __uint_as_float(coef[j][g] & 0xffff0000u);
                    top = fmaxf(top, fabsf(sc));
                    if (lane < 32) {
                        s.co[is_v][g][0][blk * 16 + (lane & 15)] = sc * odd;
                        s.co[is_v][g][1][blk * 16 + (lane & 15)] = kTwo ? fmaf(8.0f, sc, bi) : bi;
                    }
                }
            }
        }
        top = fmaxf(top, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(top), 0xB1, 0xF, 0xF, false)));
        top = fmaxf(top, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(top), 0x4E, 0xF, 0xF, false)));
        top = fmaxf(top, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(top), 0x124, 0xF, 0xF, false)));
        top = fmaxf(top, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(top), 0x128, 0xF, 0xF, false)));
        return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(top), 16));     // the lanes of V
    };

    const NibbleBits bits;
    // ---- one tile -------------------------------------------------------------
    auto compute = [&](const Tile &s, float top, int32_t base, auto masked_tag) {
        constexpr bool kMasked = decltype(masked_tag)::value;
        f32x4 x[QT][NA];
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            const int tok = a * 16 + col;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int seg = (g * 2 + (g4 >> 1)) ^ k_swizzle<D>(tok);
                const u32x2 w = *reinterpret_cast<const u32x2 *>(s.codes + tok * kRow + seg * 16 + (g4 & 1) * 8);
                const f16x8 k0 = nibbles<kTwo>(w[0], bits), k1 = nibbles<kTwo>(w[1], bits);
                const f32x4 sc = *reinterpret_cast<const f32x4 *>(&s.co[0][g][0][a * 16 + g4 * 4]);
                const f32x4 bi = *reinterpret_cast<const f32x4 *>(&s.co[0][g][1][a * 16 + g4 * 4]);
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) {
                    f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
                    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qh[qt][g][0], c, 0, 0, 0);
                    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qh[qt][g][1], c, 0, 0, 0);
                    if constexpr (kTwo) {
                        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, ql[qt][g][0], c, 0, 0, 0);
                        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, ql[qt][g][1], c, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (g == 0) x[qt][a][i] = sc[i] * c[i];
                        else x[qt][a][i] = fmaf(sc[i], c[i], x[qt][a][i]);
                        x[qt][a][i] = fmaf(bi[i], qsum[qt][g], x[qt][a][i]);
                    }
                }
            }
        }
        // exponent of a largest value scale: every scale is below 2^es
        auto exponent = [](float v) {
            const int e = static_cast<int>((__float_as_uint(v) >> 23) & 0xff) - 126;
            return static_cast<float>(e < -60 ? -60 : e > 100 ? 100 : e);
        };
        uint32_t visible[QT];                              // bit a * 4 + i
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            float m = kNoReference, scale = top;
            if constexpr (kMasked) {
                visible[qt] = 0;
                scale = 0.0f;
                const int32_t last = pos[qt] - base;
                const int64_t first = p.window > 0 ? int64_t(pos[qt]) - p.window + 1 - base : -1;
#pragma unroll
                for (int a = 0; a < NA; ++a) {
                    f32x4 sc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const f32x4 v = *reinterpret_cast<const f32x4 *>(&s.co[1][g][0][a * 16 + g4 * 4]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) sc[i] = fmaxf(sc[i], fabsf(v[i]) * (i & 1 ? 16.0f : 1.0f));
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = a * 16 + g4 * 4 + i;
                        const bool see = tok <= last && tok >= first;
                        visible[qt] |= see ? 1u << (a * 4 + i) : 0u;
                        m = see ? fmaxf(m, x[qt][a][i] * factor[qt]) : m;
                        scale = see ? fmaxf(scale, sc[i]) : scale;
                    }
                }
            } else {
                float hi = x[qt][0][0];
#pragma unroll
                for (int a = 0; a < NA; ++a)
#pragma unroll
                    for (int i = 0; i < 4; ++i) hi = fmaxf(hi, x[qt][a][i]);
                m = fmaxf(m, hi * factor[qt]);
            }
            // the reference of a row is moved by what the row sees alone, so
            // that nothing masked, and no other row, changes a bit of it
            const float want = m + (exponent(scale) - kHead);
            if (__any(want > ref[qt] + kSlack)) {
                // the four lanes of a row move together
                const float most = max_over_groups(want);
                const float next = most > ref[qt] + kSlack ? most : ref[qt];
                const float shrink = __builtin_amdgcn_exp2f(ref[qt] - next);
                ref[qt] = next;
                total[qt] *= shrink;
#pragma unroll
                for (int g = 0; g < NG; ++g) bias[qt][g] *= shrink;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) acc[qt][d] *= shrink;
            }
#pragma unroll
            for (int a = 0; a < NA; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float w = __builtin_amdgcn_exp2f(fmaf(x[qt][a][i], factor[qt], -ref[qt]));
                    if constexpr (kMasked) w = visible[qt] >> (a * 4 + i) & 1u ? w : 0.0f;
                    x[qt][a][i] = w;
                    total[qt] += w;
                }
        }
        // out += V^T w
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            __builtin_amdgcn_sched_barrier(0);               // or the operands of several groups are held at once
            f16x8 ph[QT][NST], pl[kTwo ? QT : 1][NST];
#pragma unroll
            for (int st = 0; st < NST; ++st) {
                f32x4 sc[2], bi[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sc[h] = *reinterpret_cast<const f32x4 *>(&s.co[1][g][0][(st * 2 + h) * 16 + g4 * 4]);
                    bi[h] = *reinterpret_cast<const f32x4 *>(&s.co[1][g][1][(st * 2 + h) * 16 + g4 * 4]);
                }
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) {
                    u32x4 hi, lo;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float s0 = sc[0][r], s1 = sc[1][r], b0 = bi[0][r], b1 = bi[1][r];
                        const float w0 = x[qt][st * 2][r], w1 = x[qt][st * 2 + 1][r];
                        if constexpr (kMasked) {
                            // coefficients of tokens the row does not see may be anything
                            const bool see0 = visible[qt] >> (st * 8 + r) & 1u, see1 = visible[qt] >> (st * 8 + 4 + r) & 1u;
                            s0 = see0 ? s0 : 0.0f, b0 = see0 ? b0 : 0.0f;
                            s1 = see1 ? s1 : 0.0f, b1 = see1 ? b1 : 0.0f;
                        }
                        bias[qt][g] = fmaf(w0, b0, bias[qt][g]);
                        bias[qt][g] = fmaf(w1, b1, bias[qt][g]);
                        const uint32_t pair = pack_f16(w0 * s0, w1 * s1);
                        hi[r] = pair;
                        if constexpr (kTwo) {
                            const f16x2 hh = __builtin_bit_cast(f16x2, pair);
                            lo[r] = pack_f16(fmaf(w0, s0, -static_cast<float>(hh[0])), fmaf(w1, s1, -static_cast<float>(hh[1])));
                        }
                    }
                    ph[qt][st] = __builtin_bit_cast(f16x8, hi);
                    if constexpr (kTwo) pl[qt][st] = __builtin_bit_cast(f16x8, lo);
                }
            }
            // lane `col` of group g4 addresses the codes of token
            // 16 (col / 4) + 4 g4 + col % 4 and gets channel `col` of 16 tokens
            // (32-token tiles: of 8 tokens for each of two blocks of channels)
            typedef int i32x2 __attribute__((ext_vector_type(2)));
            typedef __attribute__((address_space(3))) i32x2 *LdsPtr;
            auto transposed = [&](int chunk, int tok) {     // chunk: 8-byte piece of the token's codes
                const int seg = (chunk >> 1) ^ v_swizzle<D>(tok);
                return __builtin_amdgcn_ds_read_tr4_b64_v2i32(
                    (LdsPtr)(__attribute__((address_space(3))) void *)(s.codes + (kTok + tok) * kRow + seg * 16 + (chunk & 1) * 8));
            };
            if constexpr (kTok == 64) {
                const int tok = (col >> 2) * 16 + g4 * 4 + (col & 3);
#pragma unroll
                for (int db = 0; db < 4; ++db) {
                    const i32x2 w = transposed(g * 4 + db, tok);
#pragma unroll
                    for (int st = 0; st < NST; ++st) {
                        const f16x8 v = nibbles<kTwo>(static_cast<uint32_t>(w[st]), bits);
#pragma unroll
                        for (int qt = 0; qt < QT; ++qt) {
                            acc[qt][g * 4 + db] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, ph[qt][st], acc[qt][g * 4 + db], 0, 0, 0);
                            if constexpr (kTwo)
                                acc[qt][g * 4 + db] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pl[qt][st], acc[qt][g * 4 + db], 0, 0, 0);
                        }
                    }
                }
            } else {
                const int tok = ((col >> 2) & 1) * 16 + g4 * 4 + (col & 3);
#pragma unroll
                for (int dp = 0; dp < 2; ++dp) {
                    const i32x2 w = transposed(g * 4 + dp * 2 + (col >> 3), tok);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const f16x8 v = nibbles<kTwo>(static_cast<uint32_t>(w[h]), bits);
                        const int db = g * 4 + dp * 2 + h;
#pragma unroll
                        for (int qt = 0; qt < QT; ++qt) {
                            acc[qt][db] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, ph[qt][0], acc[qt][db], 0, 0, 0);
                            if constexpr (kTwo)
                                acc[qt][db] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pl[qt][0], acc[qt][db], 0, 0, 0);
                        }
                    }
                }
            }
        }
    };

    // positions of the first and the last row of the workgroup: a tile that
    // every row sees whole needs no masks
    const int64_t row_end = t.row0 + R < t.rows ? t.row0 + R : t.rows;
    const int64_t first_pos = int64_t(t.kv) - t.n_q + t.row0 / p.group, last_pos = int64_t(t.kv) - t.n_q + (row_end - 1) / p.group;
    auto whole = [&](int32_t base) {
        return base + kTok - 1 <= first_pos && base + kTok <= end && (p.window <= 0 || base > last_pos - p.window);
    };

    const int trips = (tiles + KW - 1) / KW;
    if (kw < tiles) {
        fetch_pages(kw);
        fetch_tile(kw);
        if (kw + KW < tiles) fetch_pages(kw + KW);
    }
    for (int i = 0; i < trips; ++i) {
        const int tile = kw + i * KW;
        const bool live = tile < tiles;
        asm volatile("" : "+v"(lane));
        col = lane & 15, g4 = lane >> 4;
        Tile &s = bufs[RW > 1 ? i & 1 : 0];
        float top = 0.0f;
        if (live) top = put_tile(s);
        if constexpr (RW > 1) {
            if (live && lane == 0) s.top[rw] = top;      // 0 from waves that fetch no coefficients
            __syncthreads();
        } else {
            // one wave's LDS operations complete in order; keep the compiler from moving them
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        if (!live) continue;
        if (tile + KW < tiles) {
            fetch_tile(tile + KW);
            if (tile + 2 * KW < tiles) fetch_pages(tile + 2 * KW);
        }
        if constexpr (RW > 1) {
#pragma unroll
            for (int w = 0; w < RW; ++w) top = fmaxf(top, s.top[w]);
        }
        const int32_t base = begin + tile * kTok;
        if (whole(base)) compute(s, top, base, MaskTag<false>{});
        else compute(s, top, base, MaskTag<true>{});
        if constexpr (RW == 1) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    }

    // ---- the wave's sums, then the groups of waves joined ---------------------
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        total[qt] = pair_sum<5>(pair_sum<4>(total[qt]));
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const float b = pair_sum<5>(pair_sum<4>(bias[qt][g]));
#pragma unroll
            for (int db = 0; db < 4; ++db) {
                acc[qt][g * 4 + db] *= 1.0f / kUnit;
                acc[qt][g * 4 + db] += b;
            }
        }
    }
    const float nan = __builtin_nanf("");
    constexpr float kLn2 = 0.693147180559945309f;
    if constexpr (KW == 1) {
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            const int64_t row = t.row0 + rw * 16 * QT + qt * 16 + col;
            if (row >= t.rows) continue;
            const int32_t tok = static_cast<int32_t>(row / p.group);
            const int head = kv_head * p.group + static_cast<int>(row - int64_t(tok) * p.group);
            const int64_t orow = int64_t(t.q0 + tok) * p.q_heads + head;
            if (p.nsplit > 1) {
                float *dst = p.part_out + (orow * p.nsplit + blockIdx.y) * D;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) *reinterpret_cast<f32x4 *>(dst + d * 16 + g4 * 4) = acc[qt][d];
                if (g4 == 0) {
                    float *st = p.part_stat + (orow * p.nsplit + blockIdx.y) * 2;
                    st[0] = ref[qt], st[1] = total[qt];
                }
            } else {
                const float inv = t.poison ? nan : total[qt] == 0.0f ? 0.0f : 1.0f / total[qt];
                T *dst = static_cast<T *>(p.out) + int64_t(t.q0 + tok) * p.out_stride + int64_t(head) * D;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) store_out4(dst + d * 16 + g4 * 4, acc[qt][d] * inv);
                if (p.lse && g4 == 0)
                    p.lse[orow] = t.poison ? nan : total[qt] == 0.0f ? -__builtin_inff()
                                                                            : (ref[qt] + __log2f(total[qt])) * kLn2;
            }
        }
    } else {
        constexpr int kPitch = D + 4;
        __syncthreads();                                   // every wave is done with its tiles
        float *mine = reinterpret_cast<float *>(lds) + static_cast<int64_t>(rw * KW + kw) * (16 * QT) * kPitch;
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            float *dst = mine + (qt * 16 + col) * kPitch;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) *reinterpret_cast<f32x4 *>(dst + d * 16 + g4 * 4) = acc[qt][d];
            if (g4 == 0) dst[D] = ref[qt], dst[D + 1] = total[qt];
        }
        __syncthreads();
        // the KW waves of a row group share its rows; 4 channels a thread
        const float *all = reinterpret_cast<const float *>(lds) + static_cast<int64_t>(rw * KW) * (16 * QT) * kPitch;
        constexpr int kQuads = D / 4;
        for (int i = kw * 64 + lane; i < 16 * QT * kQuads; i += KW * 64) {
            const int r = i / kQuads, d = (i % kQuads) * 4;
            const int64_t row = t.row0 + rw * 16 * QT + r;
            if (row >= t.rows) continue;
            float m = kNoReference, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const float rf = all[(w * 16 * QT + r) * kPitch + D];
                m = rf > m || rf != rf ? rf : m;
            }
            f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const float *src = all + (w * 16 * QT + r) * kPitch;
                const float f = __builtin_amdgcn_exp2f(src[D] - m);
                sum = fmaf(f, src[D + 1], sum);
                o += f * *reinterpret_cast<const f32x4 *>(src + d);
            }
            const int32_t tok = static_cast<int32_t>(row / p.group);
            const int head = kv_head * p.group + static_cast<int>(row - int64_t(tok) * p.group);
            const int64_t orow = int64_t(t.q0 + tok) * p.q_heads + head;
            if (p.nsplit > 1) {
                const int64_t at = orow * p.nsplit + blockIdx.y;
                *reinterpret_cast<f32x4 *>(p.part_out + at * D + d) = o;
                if (d == 0) p.part_stat[at * 2] = m, p.part_stat[at * 2 + 1] = sum;
            } else {
                const float inv = t.poison ? nan : sum == 0.0f ? 0.0f : 1.0f / sum;
                store_out4(static_cast<T *>(p.out) + int64_t(t.q0 + tok) * p.out_stride + int64_t(head) * D + d, o * inv);
                if (p.lse && d == 0)
                    p.lse[orow] = t.poison ? nan : sum == 0.0f ? -__builtin_inff() : (m + __log2f(sum)) * kLn2;
            }
        }
    }
}

// Joins the splits of a row and head: WAVES waves of a workgroup of 4 each
// (one where splits are few, four where rows are few and splits many). The
// statistics of the splits are taken a lane each; then runs of D / 4 lanes
// add up the splits s = run, run + runs, ..., and the runs are added in a
// fixed tree. The rows of a tile share their splits, so their count is found
// from the row's tile as attn_kernel does.
constexpr int kMaxSplits = 256;

template <typename T, int D, int R, int TOK, int WAVES>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnParams p)
{
    constexpr int kLanes = D / 4, kRuns = WAVES * 64 / kLanes;
    __shared__ float weight[4 / WAVES][WAVES == 1 ? 64 : kMaxSplits];
    __shared__ f32x4 sums[WAVES == 1 ? 1 : 4][kLanes];
    __shared__ float red[4][2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int mine = WAVES == 1 ? wave : 0, id = WAVES == 1 ? lane : threadIdx.x;
    const int64_t row = int64_t(blockIdx.x) * (4 / WAVES) + mine;
    if (row >= p.total_q * p.q_heads) return;              // whole waves; never with WAVES = 4
    const int64_t tok = row / p.q_heads;
    const int head = static_cast<int>(row - tok * p.q_heads);
    // the request of this query row: the last that starts at or before it
    int count = 0;
    for (int base = 0; base < p.batch; base += 64) {
        const int b = base + lane;
        const uint64_t m = __ballot(b < p.batch && attn_cu(p, b) <= tok);
        count += __popcll(m);
        if (m != ~0ull) break;
    }
    if (count == 0) return;
    RowTile t;
    t.b = count - 1;
    t.q0 = attn_cu(p, t.b);
    t.n_q = attn_cu(p, t.b + 1) - t.q0;
    if (tok - t.q0 >= t.n_q) return;
    const int64_t r = (tok - t.q0) * p.group + head % p.group;
    tile_tokens(p, t, r / R * R, R);
    const int32_t from = t.lo / TOK * TOK;
    int n = static_cast<int>((int64_t(t.hi) - from + p.chunk - 1) / p.chunk);
    n = t.hi <= from ? 0 : n < p.nsplit ? n : p.nsplit;

    const float *stat = p.part_stat + row * p.nsplit * 2;
    float m = kNoReference, own = 0.0f;
    bool bad = false;                                      // a NaN reference
    if (id < n) {
        m = stat[id * 2];
        own = stat[id * 2 + 1];
        bad = m != m;
    }
    const float ref_own = m;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, lane_xor_f32(m, d));
    bad = __any(bad);
    if constexpr (WAVES > 1) {
        if (lane == 0) red[wave][0] = bad ? __builtin_nanf("") : m;
        __syncthreads();
        m = kNoReference;
        bad = false;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float v = red[w][0];
            bad = bad || v != v;
            m = fmaxf(m, v);
        }
    }
    if (bad) m = __builtin_nanf("");
    const float f = id < n ? __builtin_amdgcn_exp2f(ref_own - m) : 0.0f;
    float sum = f * own;
    if (id < n) weight[mine][id] = f;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += lane_xor_f32(sum, d);
    if constexpr (WAVES > 1) {
        if (lane == 0) red[wave][1] = sum;
        __syncthreads();
        sum = (red[0][1] + red[1][1]) + (red[2][1] + red[3][1]);
    } else {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }

    const int run = id / kLanes, quad = id % kLanes;
    const float *part = p.part_out + row * p.nsplit * D + quad * 4;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int s = run; s < n; s += kRuns) o += weight[mine][s] * *reinterpret_cast<const f32x4 *>(part + int64_t(s) * D);
#pragma unroll
    for (int d = 32; d >= kLanes; d >>= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += lane_xor_f32(o[i], d);
    if constexpr (WAVES > 1) {
        if (lane < kLanes) sums[wave][lane] = o;
        __syncthreads();
        if (threadIdx.x >= kLanes) return;
        o = (sums[0][quad] + sums[1][quad]) + (sums[2][quad] + sums[3][quad]);
    } else if (lane >= kLanes) {
        return;
    }
    const float nan = __builtin_nanf("");
    const float inv = t.poison ? nan : sum == 0.0f ? 0.0f : 1.0f / sum;
    store_out4(static_cast<T *>(p.out) + tok * p.out_stride + int64_t(head) * D + quad * 4, o * inv);
    if (p.lse && quad == 0)
        p.lse[row] = t.poison ? nan : sum == 0.0f ? -__builtin_inff() : (m + __log2f(sum)) * 0.693147180559945309f;
}

}  // namespace qg
