// mx_gemm.hip -- entry points of the MX products: checks, choice of kernel,
// launches.
#include "mx_host.hpp"

#include <algorithm>

#include "mx_few.hpp"
#include "mx_tile.hpp"

namespace {

struct Call {
    int xfmt, act, dtype;
    bool grouped;
    int64_t M, K, N;        // N: rows, or pairs of the grouped form
    int experts;
};

// Tiles of T rows: of all rows, or at most of the experts' rows (each of
// the experts that has rows leaves one tile part empty).
int64_t row_tiles(const Call &c, int64_t T)
{
    if (!c.grouped) return ceil_div(c.N, T);
    const int64_t some = std::min<int64_t>(c.experts, c.N);
    return std::min(c.N, (c.N + some * (T - 1)) / T);
}

template <int XF, typename T, bool SILU, bool GROUPED, int MI, int KS>
void launch_few(const Call &c, qg::MxGemmParams p, hipStream_t stream)
{
    p.tiles_m = static_cast<int>(ceil_div(c.M, 16 * MI * qg::kFewWaves / KS));
    p.tiles_n = static_cast<int>(row_tiles(c, 16));
    hipLaunchKernelGGL((qg::mx_few_kernel<XF, T, SILU, GROUPED, MI, KS>), dim3(static_cast<unsigned>(int64_t(p.tiles_m) * p.tiles_n)),
                       dim3(qg::kFewThreads), 0, stream, p);
}

// Scales laid out for the tiles, in the workspace: the weights', then x's.
int64_t weight_rows(const Call &c) { return c.M * (c.act == QMX_SILU_MUL ? 2 : 1) * (c.grouped ? c.experts : 1); }
int64_t scale_stages(const Call &c) { return ceil_div(c.K, qg::kTileK); }
size_t weight_scale_bytes(const Call &c) { return align256(static_cast<size_t>(scale_stages(c)) * weight_rows(c) * qg::kTileScale); }
size_t row_scale_bytes(const Call &c) { return align256(static_cast<size_t>(scale_stages(c)) * c.N * qg::kTileScale); }
size_t tile_workspace(const Call &c, int64_t bn)
{
    return weight_scale_bytes(c) + row_scale_bytes(c) + (c.grouped ? align256(row_tiles(c, bn) * sizeof(qg::MxTileEntry)) : 0);
}
int64_t scale_workgroups(const Call &c, int64_t bn)
{
    return ceil_div(weight_rows(c), 64) + ceil_div(c.N, 64) + (c.grouped ? ceil_div(row_tiles(c, bn), qg::kScaleThreads) : 0);
}

void launch_scales(const Call &c, int bn, qg::MxGemmParams &p, void *ws, hipStream_t stream)
{
    qg::MxScalesParams s{};
    s.ws = p.ws;
    s.xs = p.xs;
    s.to_w = static_cast<uint8_t *>(ws);
    s.to_x = s.to_w + weight_scale_bytes(c);
    s.wrows = weight_rows(c);
    s.xrows = c.N;
    s.wblocks = static_cast<int32_t>(ceil_div(s.wrows, 64));
    s.pitch = p.pitch;
    s.blocks = static_cast<int32_t>(c.K / qg::kMxBlock);
    s.stages = static_cast<int32_t>(scale_stages(c));
    s.order = p.order;
    s.x_rows = p.x_rows;
    s.top = p.top;
    s.xblocks = static_cast<int32_t>(ceil_div(c.N, 64));
    s.offsets = p.offsets;
    s.experts = p.experts;
    s.tiles_n = static_cast<int32_t>(row_tiles(c, bn));
    s.bn = bn;
    s.tiles = reinterpret_cast<qg::MxTileEntry *>(s.to_x + row_scale_bytes(c));
    p.tiles = s.tiles;
    hipLaunchKernelGGL(qg::mx_scales_kernel, dim3(static_cast<unsigned>(scale_workgroups(c, bn))), dim3(qg::kScaleThreads), 0, stream, s);
    p.ws = s.to_w;
    p.xs = s.to_x;
    p.ws_rows = s.wrows;
}

template <int XF, typename T, bool SILU, bool GROUPED, int BM, int BN, int WM, int WN, int D>
void launch_tile(const Call &c, qg::MxGemmParams p, void *ws, hipStream_t stream)
{
    launch_scales(c, BN, p, ws, stream);
    p.tiles_m = static_cast<int>(ceil_div(c.M, BM / (SILU ? 2 : 1)));
    p.tiles_n = static_cast<int>(row_tiles(c, BN));
    static std::atomic<uint64_t> asked{0};
    constexpr size_t bytes = qg::MxTileLds<XF, BM, BN, WM * WN, D>::bytes;
    constexpr int64_t per = 160 * 1024 / bytes;      // workgroups that a compute unit holds
    static_assert(per >= 1, "LDS of a compute unit");
    const auto kernel = &qg::mx_tile_kernel<XF, T, SILU, GROUPED, BM, BN, WM, WN, D>;
    allow_dynamic_lds(reinterpret_cast<const void *>(kernel), bytes, asked);
    const int64_t grid = std::min(int64_t(p.tiles_m) * p.tiles_n, per * kComputeUnits);
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(64 * WM * WN), bytes, stream, p);
}

// Rows that a tile has to fill: of an expert on average in the grouped form.
int64_t usual_rows(const Call &c) { return c.grouped ? ceil_div(c.N, c.experts) : c.N; }

enum Kind { kFew16, kTile64, kTile128, kTile256 };

Kind choose(const Call &c)
{
    const int64_t rows = usual_rows(c), wide = c.M * (c.act == QMX_SILU_MUL ? 2 : 1);
    if (rows <= 16) return kFew16;
    const auto tiles = [&](int64_t bm, int64_t bn) { return ceil_div(wide, bm) * row_tiles(c, bn); };
    if (rows > 128 && tiles(256, 256) >= 2 * kComputeUnits) return kTile256;
    if (rows > 64 && tiles(128, 128) >= kComputeUnits) return kTile128;
    return kTile64;
}

// Rows of x that a tile holds.
int64_t tile_rows(const Call &c)
{
    switch (choose(c)) {
        case kFew16: return 16;
        case kTile64: return 64;
        case kTile128: return 128;
        default: return c.xfmt == QMX_E2M1 && c.act == QMX_NONE && !c.grouped ? 256 : 128;
    }
}

size_t workspace(const Call &c) { return c.N == 0 || choose(c) == kFew16 ? 0 : tile_workspace(c, tile_rows(c)); }

// Workgroups of the call's launches, and tiles (more than a launch takes are refused).
int64_t workgroups(const Call &c)
{
    const int64_t wide = c.M * (c.act == QMX_SILU_MUL ? 2 : 1);
    if (choose(c) == kFew16) return ceil_div(c.M, 16) * row_tiles(c, 16);
    return std::max(scale_workgroups(c, 64), ceil_div(wide, 64) * row_tiles(c, 64));
}

template <int XF, typename T, bool SILU, bool GROUPED>
void launch(const Call &c, const qg::MxGemmParams &p, void *ws, hipStream_t stream)
{
    switch (choose(c)) {
        case kFew16:
            // waves side by side where there are enough of them, else four to an output block
            if (ceil_div(c.M, 32) * row_tiles(c, 16) >= 4 * kComputeUnits)
                return launch_few<XF, T, SILU, GROUPED, SILU ? 1 : 2, 1>(c, p, stream);
            return launch_few<XF, T, SILU, GROUPED, 1, 4>(c, p, stream);
        case kTile64: return launch_tile<XF, T, SILU, GROUPED, 64, 64, 1, 2, 2>(c, p, ws, stream);
        case kTile128: return launch_tile<XF, T, SILU, GROUPED, 128, 128, 2, 2, 2>(c, p, ws, stream);
        default:
            if constexpr (XF == qg::kMxE2M1 && !SILU && !GROUPED)
                return launch_tile<XF, T, SILU, GROUPED, 256, 256, 2, 4, 2>(c, p, ws, stream);
            else if constexpr (XF == qg::kMxE2M1)
                return launch_tile<XF, T, SILU, GROUPED, 256, 128, 4, 2, 3>(c, p, ws, stream);
            else
                return launch_tile<XF, T, SILU, GROUPED, 256, 128, 2, 4, 2>(c, p, ws, stream);
    }
}

template <int XF, typename T>
void launch_form(const Call &c, const qg::MxGemmParams &p, void *ws, hipStream_t stream)
{
    if (c.act == QMX_SILU_MUL)
        c.grouped ? launch<XF, T, true, true>(c, p, ws, stream) : launch<XF, T, true, false>(c, p, ws, stream);
    else
        c.grouped ? launch<XF, T, false, true>(c, p, ws, stream) : launch<XF, T, false, false>(c, p, ws, stream);
}

void launch_any(const Call &c, const qg::MxGemmParams &p, void *ws, hipStream_t stream)
{
    if (c.xfmt == QMX_E2M1)
        c.dtype == QG_F32 ? launch_form<qg::kMxE2M1, float>(c, p, ws, stream) : launch_form<qg::kMxE2M1, uint16_t>(c, p, ws, stream);
    else
        c.dtype == QG_F32 ? launch_form<qg::kMxE4M3, float>(c, p, ws, stream) : launch_form<qg::kMxE4M3, uint16_t>(c, p, ws, stream);
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
    launch_any(c, params(c, x_codes, x_scales, w_codes, w_scales, y), ws, stream);
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
    launch_any(c, p, ws, stream);
    return launch_status();
}

}  // extern "C"
