// attn_common.hpp -- causal attention of new tokens over the paged 4-bit cache.
//
// Mathematics. For a query row q and tokens t with key k_t[d] =
// s_t[g] * c_t[d] + b_t[g] (g = d / 64, c the 4-bit code),
//
//   x_t = q . k_t = sum_g ( s_t[g] * sum_{d in g} q[d] c_t[d] + b_t[g] * Q[g] ),   Q[g] = sum_{d in g} q[d],
//   out[d] = ( sum_t (w_t s'_t[g]) (c'_t[d] - z) + sum_t w_t (b'_t[g] + z s'_t[g]) ) / sum_t w_t,   w_t = 2^(f x_t - R),
//
// one pass over the tokens with a reference R a row (the softmax does not
// depend on R). The codes themselves go to the matrix cores: they are exact
// in binary16, so nothing of the cache is rounded, and a float32 query or
// weight goes as two binary16 pieces (22 bits) where a dequantized cache
// would need three products of pieces. Scales and biases are applied in
// float32 outside of them. With float32 queries the codes of K and V are
// centred (z), so that the accumulators hold sums that cancel no worse than the
// result does.
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
// subnormals n * 2^-24 (bfloat16 queries) or, with an OR and a packed add, as
// c - 8 (float32 queries); odd nibbles come out 16 times too large, which the
// other operand makes good.
// V's codes are stored token by token; ds_read_b64_tr_b4 transposes 16 x 16
// nibbles among 16 lanes as it reads them.
//
// Work. The rows of a request and key/value head are its new tokens times the
// query heads that share the head, alike to the kernels. attn_few.hpp takes up
// to 32 of them (decode steps, checks of a few tokens) and gives the waves of a
// workgroup different tokens; attn_rows.hpp takes more and gives them different
// rows of the same tokens. Where there are few workgroups the tokens are cut
// into `nsplit` chunks; partial results (reference, sum, output) are joined by
// attn_join.hpp in a fixed order.
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
    int32_t window;       // 0: none
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
// The weights' products with the value scales are binary16 operands, which hold
// 2^-24 to 2^16. Tiles of tokens are taken in one of two ways.
//
// Plain tiles: every row sees all of their tokens, and their value scales lie in
// one range, 2^(E - kRange) to 2^E for an exponent E of the workgroup. A row's
// reference is 2^-kHead below its largest score times 2^E and moves only when
// that passes it by kSlack, so the accumulators are rarely rescaled: products
// stay below 2^(kHead + kSlack), and every channel group's largest one is at
// least 1 (an odd token's a 16th of it) and keeps its 21 bits. They are taken as
// they are.
//
// Careful tiles, all others: every row and group brings its products into the
// range by a power of two of its own, that of the tile's largest, and undoes it on
// the sums (about twice the vector work). They move the reference by the smallest
// scale, so that no group's products in other tiles are lost below it, unless some
// weight times its value would pass 2^(kApart + kHead + kSlack); and by what the
// row itself sees, so that nothing masked, and no other row, changes it. One that is
// careful for its scales alone sets E anew, kAbove above its largest one's.
//
// The sizes of values move a reference by 2^kSmallest to 2^kLargest at most:
// weights, their sums and those of the values stay inside of float32.
constexpr float kHead = 9.0f, kSlack = 5.0f;
constexpr int kRange = 9, kAbove = 2, kApart = 70, kSmallest = -50, kLargest = 60;
static_assert(kRange <= kHead, "a group's largest product in a plain tile is at least 2^(kHead - kRange)");

// The e of a positive v in [2^(e-1), 2^e).
__device__ __forceinline__ int float_exponent(float v) { return static_cast<int>((__float_as_uint(v) >> 23) & 0xff) - 126; }

// What a value's size counts as for the reference: its scale, or its bias where
// that is large (codes reach 15 scales).
__device__ __forceinline__ float value_size(float scale, float bias) { return fmaxf(fabsf(scale), fabsf(bias) * 0.0625f); }

// Whether a token's value scale and bias (as stored, bfloat16 bits) are in the
// range of E; NaN and infinity are not.
__device__ __forceinline__ bool in_range(uint32_t coef, int E)
{
    const uint32_t scale = (coef << 16) & 0x7fffffffu, bias = coef & 0x7fff0000u;
    return (scale - (static_cast<uint32_t>(127 + E - kRange) << 23) < (static_cast<uint32_t>(kRange) << 23)) &
           (bias < (static_cast<uint32_t>(127 + 4 + E) << 23));        // no branches
}

// The rows of one tile of query rows: request b, rows row0.. of its rows
// (row = token * group + head), and the tokens [lo, hi) that any of them sees.
struct RowTile {
    int b;
    int32_t q0;           // first query row of the request in the batch
    int32_t n_q, kv;      // its new tokens that have rows, and its tokens
    int32_t before;       // tokens before its first row's (below 0: that many rows see none)
    uint32_t row0, rows;  // below 2^31 (checked on the host)
    int32_t first, last;  // tokens of the tile's first and last row (below 0: before the request)
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

__device__ __forceinline__ void tile_tokens(const AttnParams &p, RowTile &t, uint32_t row0, int R)
{
    t.kv = p.kv_len[t.b] < 0 ? 0 : p.kv_len[t.b];
    t.poison = t.kv > p.max_kv;
    if (t.poison) t.kv = 0;
    // counted from the request's own end: rows behind total_q do not exist, but their tokens do
    const int64_t before = int64_t(t.kv) - (int64_t(p.cu_q[t.b + 1]) - t.q0);
    t.before = static_cast<int32_t>(before < -INT32_MAX ? -INT32_MAX : before);
    t.row0 = row0;
    const uint32_t group = static_cast<uint32_t>(p.group);
    t.rows = static_cast<uint32_t>(t.n_q) * group;
    const uint32_t last = row0 + R < t.rows ? row0 + R : t.rows;
    t.first = t.before + static_cast<int32_t>(row0 / group);
    t.last = t.before + static_cast<int32_t>((last - 1) / group);
    t.hi = t.last < 0 ? 0 : t.last + 1;
    const int64_t lo = p.window > 0 ? int64_t(t.first) - p.window + 1 : 0;
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
    // row starts that are not in order can make `b` a request that starts behind this slot
    const int64_t row0 = (slot - tile_start<R>(p, t.b)) * R;
    if (t.n_q <= 0 || row0 < 0 || row0 >= int64_t(t.n_q) * p.group) return false;
    tile_tokens(p, t, static_cast<uint32_t>(row0), R);
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

// Eight nibbles as c - 8 (the odd ones c - ODD): halves (0,4), (1,5)*16,
// (2,6), (3,7)*16. With the bits of 1024 set, a half is 1024 + nibble (or + 16
// nibble) exactly.
template <int ODD>
__device__ __forceinline__ f16x8 nibbles_centred(uint32_t w, const NibbleBits &k)
{
    const uint32_t v = w >> 8;
    const f16x2 even = {(_Float16)-1032.0f, (_Float16)-1032.0f};
    const f16x2 odd = {(_Float16)(-1024.0f - 16.0f * ODD), (_Float16)(-1024.0f - 16.0f * ODD)};
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
//
// Codes lie around 7.5. In sums over many tokens c - 8 would drift by half a
// code a token, against the biases' sum: so V's codes are counted from 8 for
// even tokens and from 7 for odd ones (after 20480 tokens the relative error falls from 1.1e-5 to 1.4e-6).
template <bool CENTRED, int ODD = 8>
__device__ __forceinline__ f16x8 nibbles(uint32_t w, const NibbleBits &k)
{
    if constexpr (CENTRED) return nibbles_centred<ODD>(w, k);
    else return nibbles_tiny(w);
}
constexpr int kOddCentre = 7;

// Maximum (NaN ignored) over each run of 16 lanes.
__device__ __forceinline__ float max_over_16(float v)
{
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false)));
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false)));
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xF, 0xF, false)));
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xF, 0xF, false)));
}

// Maximum (NaN ignored) over the four lanes that share l % 16.
__device__ __forceinline__ float max_over_groups(float v)
{
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
template <typename T>
__device__ __forceinline__ void store_out4(T *dst, f32x4 v);
template <>
__device__ __forceinline__ void store_out4<float>(float *dst, f32x4 v) { *reinterpret_cast<f32x4 *>(dst) = v; }
template <>
__device__ __forceinline__ void store_out4<uint16_t>(uint16_t *dst, f32x4 v)
{
    const u32x2 w = {f32_to_bf16_pair(v[0], v[1]), f32_to_bf16_pair(v[2], v[3])};
    *reinterpret_cast<u32x2 *>(dst) = w;
}

__device__ __forceinline__ float attn_inverse(const RowTile &t, float total)
{
    return t.poison ? __builtin_nanf("") : total == 0.0f ? 0.0f : 1.0f / total;
}
__device__ __forceinline__ float attn_lse(const RowTile &t, float ref, float total)
{
    return t.poison ? __builtin_nanf("")
           : total == 0.0f ? -__builtin_inff() : (ref + __log2f(total)) * 0.693147180559945309f;
}

// Exponents of the value sizes of a careful tile's tokens (up to 64), as a
// reference follows them: of the smallest scale, and of the largest value less
// kApart. Of one wave.
struct alignas(16) TileSizes {
    float low[64], top[64];
};

// Written a token a lane: `scales` and, `pitch` / 2 behind them, biases of NG
// groups, `pitch` apart. Returns the size of the token's largest value.
template <int NG>
__device__ __forceinline__ float note_sizes(TileSizes &s, const float *scales, int pitch, int token)
{
    float low = __builtin_inff(), top = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const float sc = scales[g * pitch + token] * (token & 1 ? 16.0f : 1.0f);
        low = fminf(low, fabsf(sc));
        top = fmaxf(top, value_size(sc, scales[g * pitch + pitch / 2 + token]));
    }
    int e = float_exponent(low);
    e = e < kSmallest ? kSmallest : e > kLargest ? kLargest : e;
    s.low[token] = static_cast<float>(e);
    s.top[token] = static_cast<float>(float_exponent(top) - kApart);
    return top;
}

// The range E for tokens of these sizes (one or more a lane).
__device__ __forceinline__ int choose_range(float top)
{
    const int e = float_exponent(max_over_groups(max_over_16(top))) + kAbove;
    return __builtin_amdgcn_readfirstlane(e < kSmallest ? kSmallest : e > kLargest ? kLargest : e);
}

template <bool CAREFUL>
struct CareTag {
    static constexpr bool value = CAREFUL;
};
template <int COUNT>
struct Count {
    static constexpr int value = COUNT;
};

// The query rows of a wave (QT tiles of 16, a row to the four lanes that share
// lane % 16): their operands, and the running sums of their output.
template <typename T, int D, int QT>
struct QueryRows {
    static constexpr bool kTwo = sizeof(T) == 4;           // float32: two pieces
    static constexpr int NG = D / 64;
    static constexpr float kUnit = kTwo ? 1.0f : 5.9604644775390625e-08f;       // of a code as the matrix cores see it
    f16x8 qh[QT][NG][2], ql[kTwo ? QT : 1][NG][2];
    float qsum[QT][NG], factor[QT];
    f32x4 acc[QT][D / 16];
    float ref[QT], total[QT], bias[QT][NG];

    // `pos` (LDS, 16 QT): the rows' tokens, -1 for no row or none; careful tiles
    // read them there, the others have no register for them.
    __device__ __forceinline__ void load(const AttnParams &p, const RowTile &t, int kv_head, uint32_t first, int lane, int32_t *pos)
    {
        const int col = lane & 15, g4 = lane >> 4;
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            const uint32_t row = first + qt * 16 + col;
            const bool live = row < t.rows;
            const uint32_t tok = live ? row / static_cast<uint32_t>(p.group) : 0;
            const int head = kv_head * p.group + (live ? static_cast<int>(row - tok * p.group) : 0);
            pos[qt * 16 + col] = live ? max(t.before + static_cast<int32_t>(tok), -1) : -1;
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
            ref[qt] = kNoReference;
            total[qt] = 0.0f;
#pragma unroll
            for (int g = 0; g < NG; ++g) bias[qt][g] = 0.0f;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) acc[qt][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }

    // Adds group g's share of the scores of 16 tokens (this lane: 4 of them,
    // with scales sc and biases bi): k0, k1 their codes.
    __device__ __forceinline__ void score(int qt, int g, f16x8 k0, f16x8 k1, f32x4 sc, f32x4 bi, f32x4 &x) const
    {
        f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qh[qt][g][0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qh[qt][g][1], c, 0, 0, 0);
        if constexpr (kTwo) {
            c = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, ql[qt][g][0], c, 0, 0, 0);
            c = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, ql[qt][g][1], c, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (g == 0) x[i] = sc[i] * c[i];
            else x[i] = fmaf(sc[i], c[i], x[i]);
            x[i] = fmaf(bi[i], qsum[qt][g], x[i]);
        }
    }

    // Scores of NA blocks of 16 tokens into weights, the reference and the
    // sums scaled where a score passes it. CAREFUL: `pos` is the row's token,
    // `base` the first block's first token, `sizes` (from token `at` on) what
    // note_sizes left, visible: bit a * 4 + i; else E is the range of the value scales.
    template <bool CAREFUL, int NA>
    __device__ __forceinline__ void weigh(const AttnParams &p, int qt, int32_t pos, f32x4 (&x)[NA], uint32_t &visible, const TileSizes *sizes,
                                          int at, int E, int32_t base, int g4)
    {
        float m = kNoReference, least = kNoReference, es = static_cast<float>(E);
        if constexpr (CAREFUL) {
            visible = 0;
            es = static_cast<float>(kLargest);
            const int32_t last = pos - base;
            const int32_t first = p.window > 0 ? last - p.window + 1 : -1;
#pragma unroll
            for (int a = 0; a < NA; ++a) {
                const f32x4 low = *reinterpret_cast<const f32x4 *>(&sizes->low[at + a * 16 + g4 * 4]);
                const f32x4 top = *reinterpret_cast<const f32x4 *>(&sizes->top[at + a * 16 + g4 * 4]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = a * 16 + g4 * 4 + i;
                    const bool see = tok <= last && tok >= first;
                    visible |= see ? 1u << (a * 4 + i) : 0u;
                    const float score = x[a][i] * factor[qt];
                    m = fmaxf(m, see ? score : kNoReference);
                    least = fmaxf(least, see ? score + top[i] : kNoReference);
                    es = fminf(es, see ? low[i] : static_cast<float>(kLargest));
                }
            }
        } else {
            float hi = x[0][0];
#pragma unroll
            for (int a = 0; a < NA; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) hi = fmaxf(hi, x[a][i]);
            m = fmaxf(m, hi * factor[qt]);
        }
        const float want = CAREFUL ? fmaxf(m + es, least) - kHead : m + (es - kHead);
        if (__any(want > ref[qt] + kSlack)) {
            const float most = max_over_groups(want);      // the four lanes of a row move together
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
                float w = __builtin_amdgcn_exp2f(fmaf(x[a][i], factor[qt], -ref[qt]));
                if constexpr (CAREFUL) w = visible >> (a * 4 + i) & 1u ? w : 0.0f;
                x[a][i] = w;
                total[qt] += w;
            }
    }

    // Weights of 32 tokens (two blocks; value scales sc, biases bi of this
    // lane's) as the B operand of group g's output; their biases added up.
    // CAREFUL: times a power of two that brings the row's largest product into
    // [2^12, 2^13), and `down` its inverse.
    template <bool CAREFUL>
    __device__ __forceinline__ void pieces(int qt, int g, f32x4 w0, f32x4 w1, uint32_t visible, const f32x4 (&sc)[2],
                                           const f32x4 (&bi)[2], f16x8 &ph, f16x8 &pl, float &down)
    {
        const f32x4 s0 = sc[0], s1 = sc[1];
        float up = 1.0f;
        if constexpr (CAREFUL) {
            // the products first: the power of two alone may leave what the weights can take
            float top = 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                // coefficients of tokens the row does not see may be anything
                const bool see0 = visible >> r & 1u, see1 = visible >> (4 + r) & 1u;
                bias[qt][g] = fmaf(w0[r], see0 ? bi[0][r] : 0.0f, bias[qt][g]);
                bias[qt][g] = fmaf(w1[r], see1 ? bi[1][r] : 0.0f, bias[qt][g]);
                w0[r] *= see0 ? s0[r] : 0.0f;
                w1[r] *= see1 ? s1[r] : 0.0f;
                top = fmaxf(top, fmaxf(fabsf(w0[r]), fabsf(w1[r])));
            }
            top = max_over_groups(top);
            int e = static_cast<int>((__float_as_uint(top) >> 23) & 0xff);
            e = e < 13 ? 13 : e > 254 ? 254 : e;
            up = __uint_as_float(static_cast<uint32_t>(127 + 12 + 127 - e) << 23);
            down = __uint_as_float(static_cast<uint32_t>(127 - 12 - 127 + e) << 23);
        }
        u32x4 hi, lo;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float u0 = CAREFUL ? up : s0[r], u1 = CAREFUL ? up : s1[r];
            if constexpr (!CAREFUL) {
                bias[qt][g] = fmaf(w0[r], bi[0][r], bias[qt][g]);
                bias[qt][g] = fmaf(w1[r], bi[1][r], bias[qt][g]);
            }
            const uint32_t pair = pack_f16(w0[r] * u0, w1[r] * u1);
            hi[r] = pair;
            if constexpr (kTwo) {
                const f16x2 hh = __builtin_bit_cast(f16x2, pair);
                lo[r] = pack_f16(fmaf(w0[r], u0, -static_cast<float>(hh[0])), fmaf(w1[r], u1, -static_cast<float>(hh[1])));
            }
        }
        ph = __builtin_bit_cast(f16x8, hi);
        if constexpr (kTwo) pl = __builtin_bit_cast(f16x8, lo);
    }

    // 16 channels of output added to c: v the codes of 32 tokens.
    __device__ __forceinline__ f32x4 product(f16x8 v, f16x8 ph, f16x8 pl, f32x4 c) const
    {
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, ph, c, 0, 0, 0);
        if constexpr (kTwo) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pl, c, 0, 0, 0);
        return c;
    }
    // Channels 16 db.. of the output: N operands of 32 tokens each.
    template <bool CAREFUL, int N>
    __device__ __forceinline__ void add(int qt, int db, const f16x8 (&v)[N], const f16x8 *ph, const f16x8 *pl, float down)
    {
        if constexpr (CAREFUL) {
            f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int n = 0; n < N; ++n) c = product(v[n], ph[n], pl[n], c);
            acc[qt][db] = __builtin_elementwise_fma(c, f32x4{down, down, down, down}, acc[qt][db]);
            asm("" : "+v"(acc[qt][db]));                   // kept as four registers in a row, as the matrix cores take them
        } else {
#pragma unroll
            for (int n = 0; n < N; ++n) acc[qt][db] = product(v[n], ph[n], pl[n], acc[qt][db]);
        }
    }

    // The lanes' sums joined, the biases added to the outputs.
    __device__ __forceinline__ void close()
    {
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            total[qt] = pair_sum<5>(pair_sum<4>(total[qt]));
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float b = pair_sum<5>(pair_sum<4>(bias[qt][g]));
#pragma unroll
                for (int db = 0; db < 4; ++db) {
                    if constexpr (!kTwo) acc[qt][g * 4 + db] *= 1.0f / kUnit;
                    acc[qt][g * 4 + db] += b;
                }
            }
        }
    }

    // Results of a split, or of the whole call.
    __device__ __forceinline__ void write(const AttnParams &p, const RowTile &t, int kv_head, uint32_t first, int lane) const
    {
        const int col = lane & 15, g4 = lane >> 4;
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            const uint32_t row = first + qt * 16 + col;
            if (row >= t.rows) continue;
            const uint32_t tok = row / static_cast<uint32_t>(p.group);
            const int head = kv_head * p.group + static_cast<int>(row - tok * p.group);
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
                const float inv = attn_inverse(t, total[qt]);
                T *dst = static_cast<T *>(p.out) + int64_t(t.q0 + tok) * p.out_stride + int64_t(head) * D;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) store_out4(dst + d * 16 + g4 * 4, acc[qt][d] * inv);
                if (p.lse && g4 == 0) p.lse[orow] = attn_lse(t, ref[qt], total[qt]);
            }
        }
    }
};

// This split's tokens [begin, end) of a tile of rows; false: none, and not
// the split that writes the results of rows without tokens.
__device__ __forceinline__ bool split_tokens(const AttnParams &p, const RowTile &t, int tile, int32_t &begin, int32_t &end)
{
    const int64_t b = int64_t(t.lo / tile * tile) + int64_t(blockIdx.y) * p.chunk;
    begin = b < t.hi ? static_cast<int32_t>(b) : t.hi;
    end = t.hi - begin < p.chunk ? t.hi : begin + p.chunk;
    return begin < end || blockIdx.y == 0;
}

// Whether every row of the tile sees all of `count` tokens from `base` on.
__device__ __forceinline__ bool all_visible(const AttnParams &p, const RowTile &t, int32_t base, int count)
{
    return base + count - 1 <= t.first && (p.window <= 0 || base > t.last - p.window);
}

// Coefficients of a token's groups (scale low, bias high).
template <int NG>
__device__ __forceinline__ void load_coefs(const uint8_t *src, uint32_t (&c)[NG])
{
    if constexpr (NG == 1) {
        c[0] = *reinterpret_cast<const uint32_t *>(src);
    } else if constexpr (NG == 2) {
        const u32x2 v = *reinterpret_cast<const u32x2 *>(src);
        c[0] = v[0], c[1] = v[1];
    } else {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(src);
#pragma unroll
        for (int g = 0; g < NG; ++g) c[g] = v[g];
    }
}

// What they count as (where they are used, so that no load is waited for before):
// `known`: the token's page is in the cache, `inside`: it is one of the request's
// tokens.
__device__ __forceinline__ uint32_t coef_of(uint32_t c, bool known, bool inside)
{
    if (!known) c = 0x7fc07fc0u;             // a page outside the cache reads as NaN
    return inside ? c : 0;                   // places behind the last token hold anything
}

typedef int i32x2 __attribute__((ext_vector_type(2)));

// 16 x 16 nibbles transposed among 16 lanes: lane i addresses row i (8 bytes),
// and gets nibble i of every row.
__device__ __forceinline__ i32x2 read_transposed(const uint8_t *row)
{
    typedef __attribute__((address_space(3))) i32x2 *LdsPtr;
    return __builtin_amdgcn_ds_read_tr4_b64_v2i32((LdsPtr)(__attribute__((address_space(3))) void *)(row));
}

// One wave's LDS operations complete in order; this keeps the compiler from
// moving reads of what other lanes wrote ahead of the writes.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

}  // namespace qg
