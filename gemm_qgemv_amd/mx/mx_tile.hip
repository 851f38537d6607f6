// mx_tile.hip -- launches of the MX products for many rows.
#include "mx_call.hpp"
#include "mx_tile.hpp"

namespace qg {

namespace {

// Scales laid out for the tiles, in the workspace: the weights', then x's.
int64_t weight_rows(const MxCall &c) { return c.wide() * (c.grouped ? c.experts : 1); }
int64_t scale_stages(const MxCall &c) { return ceil_div(c.K, kTileK); }
size_t weight_scale_bytes(const MxCall &c) { return align256(static_cast<size_t>(scale_stages(c)) * weight_rows(c) * kTileScale); }
size_t row_scale_bytes(const MxCall &c) { return align256(static_cast<size_t>(scale_stages(c)) * c.N * kTileScale); }
// grouped: the list of tiles and their number, and behind it where the sorted rows' codes begin
int64_t tile_list(const MxCall &c, int64_t bn) { return static_cast<int64_t>(align256((c.row_tiles(bn) + 1) * sizeof(MxTileEntry)) / sizeof(MxTileEntry)); }
int64_t scale_workgroups(const MxCall &c, int64_t bn)
{
    return ceil_div(weight_rows(c), 64) + ceil_div(c.N, 64) + (c.grouped ? ceil_div(c.row_tiles(bn), kScaleThreads) : 0);
}

void launch_scales(const MxCall &c, int bn, MxGemmParams &p, void *ws, hipStream_t stream)
{
    MxScalesParams s{};
    s.ws = p.ws;
    s.xs = p.xs;
    s.to_w = static_cast<uint8_t *>(ws);
    s.to_x = s.to_w + weight_scale_bytes(c);
    s.wrows = weight_rows(c);
    s.xrows = c.N;
    s.wblocks = static_cast<int32_t>(ceil_div(s.wrows, 64));
    s.pitch = p.pitch;
    s.blocks = static_cast<int32_t>(c.K / kMxBlock);
    s.stages = static_cast<int32_t>(scale_stages(c));
    s.order = p.order;
    s.x_rows = p.x_rows;
    s.top = p.top;
    s.xblocks = static_cast<int32_t>(ceil_div(c.N, 64));
    s.offsets = p.offsets;
    s.experts = p.experts;
    s.tiles_n = static_cast<int32_t>(c.row_tiles(bn));
    s.bn = bn;
    s.tiles = reinterpret_cast<MxTileEntry *>(s.to_x + row_scale_bytes(c));
    p.tiles = s.tiles;
    s.x_at = reinterpret_cast<uint32_t *>(s.tiles + (c.grouped ? tile_list(c, bn) : 0));
    s.xrb = static_cast<int32_t>(mx_row_bytes(c.xfmt, c.K));
    p.x_at = s.x_at;
    hipLaunchKernelGGL(mx_scales_kernel, dim3(static_cast<unsigned>(scale_workgroups(c, bn))), dim3(kScaleThreads), 0, stream, s);
    p.ws = s.to_w;
    p.xs = s.to_x;
    p.ws_rows = s.wrows;
}

template <typename F, int BM, int BN, int WM, int WN>
void launch(const MxCall &c, MxGemmParams p, void *ws, hipStream_t stream)
{
    launch_scales(c, BN, p, ws, stream);
    p.tiles_m = static_cast<int>(ceil_div(c.M, BM / (F::SILU ? 2 : 1)));
    p.tiles_n = static_cast<int>(c.row_tiles(BN));
    static std::atomic<uint64_t> asked{0};
    constexpr size_t bytes = MxTileLds<F::XF, F::GROUPED, BM, BN, WM * WN>::bytes;
    constexpr int64_t per = 160 * 1024 / bytes;      // workgroups that a compute unit holds
    static_assert(per >= 1, "LDS of a compute unit");
    const auto kernel = &mx_tile_kernel<F::XF, typename F::T, F::SILU, F::GROUPED, BM, BN, WM, WN>;
    allow_dynamic_lds(reinterpret_cast<const void *>(kernel), bytes, asked);
    const int64_t grid = std::min(int64_t(p.tiles_m) * p.tiles_n, per * kComputeUnits);
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(64 * WM * WN), bytes, stream, p);
}

}  // namespace

int64_t mx_tile_rows(const MxCall &c, int size)
{
    return size == 256 && c.xfmt != QMX_E2M1 ? 128 : size;
}

size_t mx_tile_workspace(const MxCall &c, int size)
{
    return weight_scale_bytes(c) + row_scale_bytes(c) +
           (c.grouped ? tile_list(c, mx_tile_rows(c, size)) * sizeof(MxTileEntry) + align256(c.N * 4) : 0);
}

int64_t mx_tile_workgroups(const MxCall &c, int size)
{
    const int64_t rows = mx_tile_rows(c, size);
    return std::max(scale_workgroups(c, rows), ceil_div(c.wide(), size) * c.row_tiles(rows));
}

void mx_launch_tile(const MxCall &c, const MxGemmParams &p, int size, void *ws, hipStream_t stream)
{
    mx_dispatch(c, [&](auto form) {
        using F = decltype(form);
        if (size == 64) return launch<F, 64, 64, 1, 2>(c, p, ws, stream);
        if constexpr (F::XF == kMxE2M1)
            if (size == 128) return launch<F, 128, 128, 2, 2>(c, p, ws, stream);
        // (of e4m3 rows two slots for 256 x 256 would not fit in LDS)
        launch<F, 256, F::XF == kMxE4M3 ? 128 : 256, 2, 4>(c, p, ws, stream);
    });
}

}  // namespace qg
