// mx_gemm.hip -- entry points of the MX products: checks and the choice of the
// kernel.
#include "mx_call.hpp"

namespace {

using Call = qg::MxCall;

// Which kernel a call takes.
struct Choice {
    enum Kind { kFew, kMid, kTile } kind;
    int size;        // kFew: waves side by side or not; kMid: blocks of weight rows; kTile: weight rows
    int blocks;      // kMid: blocks of 16 rows
};

// Rows that a tile has to fill: of an expert on average in the grouped form.
int64_t usual_rows(const Call &c) { return c.grouped ? ceil_div(c.N, c.experts) : c.N; }

Choice choose(const Call &c)
{
    const int64_t rows = usual_rows(c);
    if (rows <= 16) return {Choice::kFew, ceil_div(c.M, 32) * c.row_tiles(16) >= 4 * kComputeUnits, 0};
    if (rows <= 128) {
        const int nj = rows <= 32 ? 2 : rows <= 64 ? 4 : rows <= 96 ? 6 : 8;
        return {Choice::kMid, ceil_div(c.wide(), 128) * c.row_tiles(16 * nj) >= kComputeUnits ? 4 : 2, nj};
    }
    const auto tiles = [&](int size) { return ceil_div(c.wide(), size) * c.row_tiles(qg::mx_tile_rows(c, size)); };
    if (tiles(256) >= 2 * kComputeUnits) return {Choice::kTile, 256, 0};
    if (tiles(128) >= kComputeUnits) return {Choice::kTile, 128, 0};
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
    if (k.kind == Choice::kFew) return ceil_div(c.M, 16) * c.row_tiles(16);
    if (k.kind == Choice::kMid) return ceil_div(c.wide(), 32 * k.size) * c.row_tiles(16 * k.blocks);
    return qg::mx_tile_workgroups(c, k.size);
}

void launch(const Call &c, const qg::MxGemmParams &p, void *ws, hipStream_t stream)
{
    const Choice k = choose(c);
    switch (k.kind) {
        case Choice::kFew: return qg::mx_launch_few(c, p, k.size != 0, stream);
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
