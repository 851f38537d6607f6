// mx_gemm.hip -- entry points of the MX products: checks and the choice of the
// kernel.
#include "mx_call.hpp"

namespace {

using Call = qg::MxCall;

// Which kernel a call takes.
struct Choice {
    enum Kind { kFew, kMid, kTile } kind;
    int size;        // kFew, kMid: blocks of 16 weight rows a wave takes (kFew: of outputs); kTile: weight rows
    int blocks;      // kFew: waves that split K; kMid: blocks of 16 rows
};

// Rows that a tile has to fill: of an expert on average in the grouped form.
int64_t usual_rows(const Call &c) { return c.grouped ? ceil_div(c.N, c.experts) : c.N; }

// Measured, e4m3 rows (e2m1 in brackets), outputs x K x rows:
//  few against mid     2048 x 8192 x 24: 10 against 19 us [7.6, 17]; 6144 x 2048 x 60:
//                      12, 11 [9, 8]; 17408 x 5120 x 24: 32, 21 [22, 18]
//  few against tiles   1024 x 2048 x 256: 9, 17.5 [7.5, 12]; 2048 x 8192 x 200: 45, 51 [33, 29]
//                      (6.5 pieces a compute unit: tiles of both, though e4m3 rows still
//                      do better in pieces there; the limit is one for both)
//  few of one block of outputs a wave against two   2048 x 8192 x 16: 9.3, 11.4 [7.4, 9.6];
//                      17408 x 5120 x 16: 21, 18 [15, 15]; 151936 x 2048 x 1: 33, 30 [28, 26];
//                      2048 x 8192 x 77: 21, 19 [16, 16]
//  mid against tiles   17408 x 5120 x 60: 34, 45 [21, 27]; x 90: 45, 45 [24, 28]
//  mid of 64 weight rows a wave pair against 128   6144 x 2048 x 60: 11, 15 [8, 11];
//                      17408 x 5120 x 77: 45, 37 [27, 22]
//  tiles of 64, 128 and 256 (of e4m3 256 x 128), and how full the rounds of the last are
//                      17408 x 5120 x 120: 45, 50, 63 at 27% [25, 26, 34 at 27%]
//                      6144 x 2048 x 1000: 39, 43, 33 at 75% [22, 19, 25 at 38%]
//                      6144 x 2048 x 4000: 127, 117, 83 at 100% [54, 42, 45 at 75%]
//                      17408 x 5120 x 2048: 415, 381, 290 at 85% [164, 121, 135 at 71%]
//                      5120 x 17408 x 512: 125, 139, 180 at 31% [63, 65, 112 at 16%]
Choice choose(const Call &c)
{
    const int64_t rows = usual_rows(c), wide = c.wide();
    // Workgroups of 16 outputs x 16 rows whose waves split K: for 16 rows, and
    // wherever they are few, since larger ones would leave compute units idle (the
    // weights that several read come from the caches).
    if (rows <= 16 || ceil_div(wide, 16) * c.row_tiles(16) <= 4 * kComputeUnits) {
        // as many waves share outputs as have a run of inputs each; two blocks of
        // outputs a wave once every compute unit gets a workgroup of four such waves
        const int64_t runs = ceil_div(c.K, 512);
        return {Choice::kFew, c.act == QMX_NONE && ceil_div(c.M, 32) * c.row_tiles(16) >= kComputeUnits ? 2 : 1, runs > 2 ? 4 : runs > 1 ? 2 : 1};
    }
    // The weights straight to registers, while x's rows are one tile: 128 weight rows a
    // workgroup once those of 64 are more than the compute units.
    if (rows <= 96) {
        const int nj = rows <= 32 ? 2 : rows <= 64 ? 4 : 6;
        if (ceil_div(wide, 64) * c.row_tiles(16 * nj) <= kComputeUnits) return {Choice::kMid, 2, nj};
        const int most = qg::mx_mid_most(c.xfmt);
        if (rows <= 16 * most) return {Choice::kMid, 4, std::min(nj, most)};
    }
    // The largest tiles where their rounds over the compute units are full enough for what
    // they save to show (in the grouped form half of an expert's last tile is empty).
    const auto tiles = [&](int size) {
        const int64_t T = qg::mx_tile_rows(c, size), some = std::min<int64_t>(c.experts, c.N);
        return ceil_div(wide, size) * (c.grouped ? std::min(c.N, ceil_div(c.N, T) + some / 2) : ceil_div(c.N, T));
    };
    const bool e2m1 = c.xfmt == QMX_E2M1;
    if (tiles(256) * 100 >= round_up(tiles(256), kComputeUnits) * (e2m1 ? 80 : 65)) return {Choice::kTile, 256, 0};
    if (e2m1 && tiles(128) >= kComputeUnits) return {Choice::kTile, 128, 0};
    return {Choice::kTile, 64, 0};
}

size_t workspace(const Call &c)
{
    if (c.N == 0) return 0;
    const Choice k = choose(c);
    return k.kind == Choice::kTile ? qg::mx_tile_workspace(c, k.size) : 0;
}

// Workgroups of the call's launches, and tiles (more than a launch takes are refused).
int64_t workgroups(const Call &c)
{
    const Choice k = choose(c);
    if (k.kind == Choice::kFew) return ceil_div(c.M, 64 * k.size / k.blocks) * c.row_tiles(16);
    if (k.kind == Choice::kMid) return ceil_div(c.wide(), 32 * k.size) * c.row_tiles(16 * k.blocks);
    return qg::mx_tile_workgroups(c, k.size);
}

void launch(const Call &c, const qg::MxGemmParams &p, void *ws, hipStream_t stream)
{
    const Choice k = choose(c);
    switch (k.kind) {
        case Choice::kFew: return qg::mx_launch_few(c, p, k.size, k.blocks, stream);
        case Choice::kMid: return qg::mx_launch_mid(c, p, k.size, k.blocks, stream);
        default: return qg::mx_launch_tile(c, p, k.size, ws, stream);
    }
}

bool sizes_ok(const Call &c)
{
    return mx_k_ok(c.K) && c.M >= 1 && c.M <= QMX_MAX_M && c.N >= 0 && c.N <= 0x7fffffffLL && (c.N == 0 || workgroups(c) <= kMaxWorkgroups);
}

bool kinds_ok(const Call &c)
{
    return known_mx(c.xfmt) && known_dtype(c.dtype) && (c.act == QMX_NONE || c.act == QMX_SILU_MUL);
}

// The operands, and the workspace `work` of the size that the call needs.
int check_product(const Call &c, const void *xc, const void *xs, const void *wc, const void *ws, const void *y, const void *work,
                  size_t work_bytes)
{
    if (!xc || !xs || !wc || !ws || !y) return QG_ERR_NULL;
    if (!kinds_ok(c)) return QG_ERR_FORMAT;
    if (!sizes_ok(c)) return QG_ERR_SHAPE;
    for (const void *q : {xc, wc, y})
        if (!aligned(q, kAlign)) return QG_ERR_ALIGN;
    for (const void *q : {xs, ws})
        if (!aligned(q, 4)) return QG_ERR_ALIGN;
    if (workspace(c) > 0) {
        if (!work || work_bytes < workspace(c)) return QG_ERR_WORKSPACE;
        if (!aligned(work, kAlign)) return QG_ERR_ALIGN;
    }
    return QG_OK;
}

qg::MxGemmParams params(const Call &c, const void *xc, const void *xs, const void *wc, const void *ws, void *y)
{
    qg::MxGemmParams p{};
    p.xc = static_cast<const uint8_t *>(xc);
    p.xs = static_cast<const uint8_t *>(xs);
    p.wc = static_cast<const uint8_t *>(wc);
    p.ws = static_cast<const uint8_t *>(ws);
    p.y = y;
    p.M = c.M;
    p.N = c.N;
    p.K = static_cast<int32_t>(c.K);
    p.pitch = static_cast<int32_t>(qg::mx_pitch(c.K));
    return p;
}

}  // namespace

extern "C" {

size_t qmx_gemm_workspace_bytes(int xfmt, int act, int64_t M, int64_t K, int64_t N)
{
    const Call c{xfmt, act, QG_F32, false, M, K, N, 0};
    return kinds_ok(c) && sizes_ok(c) ? workspace(c) : 0;
}

size_t qmoe_gemm_workspace_bytes(int xfmt, int act, int64_t rows, int experts, int top, int64_t M, int64_t K)
{
    if (!moe_sizes_ok(rows, experts, top)) return 0;
    const Call c{xfmt, act, QG_F32, true, M, K, rows * top, experts};
    return kinds_ok(c) && sizes_ok(c) ? workspace(c) : 0;
}

int qmx_gemm(int xfmt, const void *x_codes, const void *x_scales, const void *w_codes, const void *w_scales, int act, int dtype,
             void *y, int64_t M, int64_t K, int64_t N, void *ws, size_t ws_bytes, hipStream_t stream)
{
    const Call c{xfmt, act, dtype, false, M, K, N, 0};
    int st = check_product(c, x_codes, x_scales, w_codes, w_scales, y, ws, ws_bytes);
    if (st != QG_OK || N == 0) return st;
    const int64_t wide = M * (act == QMX_SILU_MUL ? 2 : 1), pitch = qg::mx_pitch(K);
    const Range in[4] = {range_of(x_codes, N * mx_row_bytes(xfmt, K)), range_of(x_scales, N * pitch), range_of(w_codes, wide * (K / 2)),
                         range_of(w_scales, wide * pitch)};
    const Range out[2] = {range_of(y, N * M * (dtype == QG_F32 ? 4 : 2)), range_of(ws, static_cast<int64_t>(workspace(c)))};
    st = check_alias(in, 4, out, 2);
    if (st != QG_OK) return st;

    (void)hipGetLastError();
    launch(c, params(c, x_codes, x_scales, w_codes, w_scales, y), ws, stream);
    return launch_status();
}

int qmoe_gemm(int xfmt, const void *x_codes, const void *x_scales, const void *w_codes, const void *w_scales, const int32_t *offsets,
              const int32_t *order, int64_t rows, int experts, int top, int act, int dtype, void *y, int64_t M, int64_t K, void *ws,
              size_t ws_bytes, hipStream_t stream)
{
    if (!offsets) return QG_ERR_NULL;
    if (!moe_sizes_ok(rows, experts, top)) return QG_ERR_SHAPE;
    const Call c{xfmt, act, dtype, true, M, K, rows * top, experts};
    // rows that are gathered are reached by 32-bit offsets from the first
    if (order && kinds_ok(c) && mx_k_ok(K) && rows * mx_row_bytes(xfmt, K) > 0x7fffffffLL) return QG_ERR_SHAPE;
    int st = check_product(c, x_codes, x_scales, w_codes, w_scales, y, ws, ws_bytes);
    if (st != QG_OK) return st;
    const int64_t x_rows = order ? rows : c.N;
    if (!aligned(offsets, 4) || !aligned(order, 4)) return QG_ERR_ALIGN;
    if (c.N == 0) return QG_OK;
    const int64_t wide = int64_t(experts) * M * (act == QMX_SILU_MUL ? 2 : 1), pitch = qg::mx_pitch(K);
    const Range in[6] = {range_of(x_codes, x_rows * mx_row_bytes(xfmt, K)), range_of(x_scales, x_rows * pitch),
                         range_of(w_codes, wide * (K / 2)), range_of(w_scales, wide * pitch), range_of(offsets, (int64_t(experts) + 1) * 4),
                         range_of(order, order ? c.N * 4 : 0)};
    const Range out[2] = {range_of(y, c.N * M * (dtype == QG_F32 ? 4 : 2)), range_of(ws, static_cast<int64_t>(workspace(c)))};
    st = check_alias(in, 6, out, 2);
    if (st != QG_OK) return st;

    (void)hipGetLastError();
    qg::MxGemmParams p = params(c, x_codes, x_scales, w_codes, w_scales, y);
    p.offsets = offsets;
    p.order = order;
    p.experts = experts;
    p.x_rows = x_rows;
    p.top = qg::fast_div(static_cast<uint32_t>(top));
    launch(c, p, ws, stream);
    return launch_status();
}

}  // extern "C"
